// Epilogue of the W8A8 linear layer: y = bf16( act(acc + bias[n]) + residual[m, n] ),
// every step in fp32 and one rounding to bf16 at the end.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

namespace fgfp8 {

// Values of the C header's fgfp8_act.
enum : int { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4 };

struct EpiArgs {
  const void* bias;                  // [N] bf16 or fp32, or nullptr
  const __nv_bfloat16* residual;     // [M, N] with row stride ld_r, or nullptr
  uint64_t ld_r;
  int bias_f32;
  int act;
};

// x / (1 + exp(-z)) with the hardware exponential and divide (a few fp32
// ulps, far below the bf16 step of the result).  exp(-z) = +inf gives -0.
__device__ __forceinline__ float times_sigmoid(float x, float z) { return __fdividef(x, 1.0f + __expf(-z)); }

// silu(x)      = x sigmoid(x)
// gelu_tanh(x) = x/2 (1 + tanh(c)) = x sigmoid(2 c), c = sqrt(2/pi) (x + 0.044715 x^3): the
//                sigmoid form keeps the relative accuracy of the negative tail
// gelu(x)      = x Phi(x), with Phi(-|x|) = erfc(|x| / sqrt 2) / 2 and erfc(z) = e^(-z^2) P(t),
//                t = 1 / (1 + 0.3275911 z) (Abramowitz & Stegun, 7.1.26; |error| <= 1.5e-7)
// A NaN stays a NaN in each of them.
__device__ __forceinline__ float act_gelu(float x) {
  const float z = fabsf(x) * 0.70710678118654752f;
  const float t = __fdividef(1.0f, fmaf(0.3275911f, z, 1.0f));
  float q = fmaf(1.061405429f, t, -1.453152027f);
  q = fmaf(q, t, 1.421413741f);
  q = fmaf(q, t, -0.284496736f);
  q = fmaf(q, t, 0.254829592f);
  const float phi = 0.5f * q * t * __expf(-z * z);     // Phi(-|x|)
  return x < 0.0f ? x * phi : x - x * phi;
}

__device__ __forceinline__ float apply_act(float x, int act) {
  switch (act) {
    case kActRelu: return x < 0.0f ? 0.0f : x;
    case kActSilu: return times_sigmoid(x, x);
    case kActGelu: return act_gelu(x);
    case kActGeluTanh: return times_sigmoid(x, 1.5957691216057308f * fmaf(0.044715f * x * x, x, x));
    default: return x;
  }
}

// act over 8 values, the choice made once.
__device__ __forceinline__ void apply_act8(float (&x)[8], int act) {
  switch (act) {
    case kActRelu:
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = apply_act(x[i], kActRelu);
      break;
    case kActSilu:
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = apply_act(x[i], kActSilu);
      break;
    case kActGelu:
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = apply_act(x[i], kActGelu);
      break;
    case kActGeluTanh:
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = apply_act(x[i], kActGeluTanh);
      break;
    default: break;
  }
}

// 8 accumulators of columns n.. n+7 (n % 8 == 0) with the bias, the activation
// and 8 residual values (bf16, zeros when there are none), rounded to bf16.
__device__ __forceinline__ uint4 epilogue8(float (&x)[8], const EpiArgs& e, uint64_t n, const uint4& res) {
  if (e.bias != nullptr) {
    if (e.bias_f32) {
      const float4* b = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(e.bias) + n);
      const float4 b0 = __ldg(b), b1 = __ldg(b + 1);
      x[0] += b0.x, x[1] += b0.y, x[2] += b0.z, x[3] += b0.w;
      x[4] += b1.x, x[5] += b1.y, x[6] += b1.z, x[7] += b1.w;
    } else {
      const uint4 b = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(e.bias) + n));
      const uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] += __uint_as_float(w[i] << 16);
        x[2 * i + 1] += __uint_as_float(w[i] & 0xFFFF0000u);
      }
    }
  }
  apply_act8(x, e.act);
  uint4 v;
  const uint32_t r[4] = {res.x, res.y, res.z, res.w};
  uint32_t* o = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h =
        __floats2bfloat162_rn(x[2 * i] + __uint_as_float(r[i] << 16), x[2 * i + 1] + __uint_as_float(r[i] & 0xFFFF0000u));
    o[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return v;
}

// 8 residual values of row m at column n, or zeros.
__device__ __forceinline__ uint4 load_residual8(const EpiArgs& e, uint64_t m, uint64_t n) {
  if (e.residual == nullptr) return make_uint4(0, 0, 0, 0);
  return *reinterpret_cast<const uint4*>(e.residual + m * e.ld_r + n);
}

__device__ __forceinline__ float load_bias(const EpiArgs& e, uint64_t n) {
  if (e.bias == nullptr) return 0.0f;
  return e.bias_f32 ? __ldg(reinterpret_cast<const float*>(e.bias) + n)
                    : __bfloat162float(__ldg(reinterpret_cast<const __nv_bfloat16*>(e.bias) + n));
}

}  // namespace fgfp8
