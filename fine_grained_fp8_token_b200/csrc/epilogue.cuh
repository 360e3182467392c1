// Epilogue of the W8A8 linear layer: y = bf16( act(acc + bias[n]) + residual[m, n] ),
// every step in fp32 and one rounding to bf16 at the end.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "ptx.cuh"

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

// One instruction each: 2^x and 1/x to about an ulp, subnormals as zeros.
__device__ __forceinline__ float fast_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// x / (1 + exp(-z)), two at a time in packed fp32 arithmetic.  For z < 0 the
// rounding of the exponential's argument passes into the result, |z| 2^-24
// relative, and below z = -87.3 the reciprocal of a sum past 2^126 is flushed to
// zero, so that results under |x| 2^-126 are zeros; both are far below the bf16
// step of anything that is added to them.
__device__ __forceinline__ float2 times_sigmoid2(float2 x, float2 z) {
  const float2 a = __fmul2_rn(z, make_float2(-1.44269504f, -1.44269504f));
  const float2 d = __fadd2_rn(make_float2(fast_ex2(a.x), fast_ex2(a.y)), make_float2(1.0f, 1.0f));
  return __fmul2_rn(x, make_float2(fast_rcp(d.x), fast_rcp(d.y)));
}
__device__ __forceinline__ float times_sigmoid(float x, float z) {
  return times_sigmoid2(make_float2(x, x), make_float2(z, z)).x;
}

// silu(x)      = x sigmoid(x)
// gelu_tanh(x) = x/2 (1 + tanh(c)) = x sigmoid(2 c), c = sqrt(2/pi) (x + 0.044715 x^3): the
//                sigmoid form keeps the relative accuracy of the negative tail
// gelu(x)      = x Phi(x) = max(x, 0) - |x| Phi(-|x|), with Phi(-a) = e^(-a^2 / 2) Q(t),
//                t = 1 / (1 + 0.36 a), Q of degree 7 without a constant term: a fit of
//                e^(a^2 / 2) erfc(a / sqrt 2) / 2 over 0 <= a <= 14 with the least largest
//                relative error (9e-7), found by Lawson's weighted least squares.  The
//                exponential's argument adds up to 2^-17 in the far tail.  Relative, as the
//                negative tail is all of the result there: a fit with 1.5e-7 absolute error
//                was off by 0.4% at x = -6.  Beyond a = 64 Phi(-a) is 0 in fp32
// A NaN stays a NaN in each of them.
__device__ __forceinline__ float2 gelu2(float2 x) {
  auto both = [](float v) { return make_float2(v, v); };
  const float2 a = make_float2(fminf(fabsf(x.x), 64.0f), fminf(fabsf(x.y), 64.0f));
  const float2 d = __ffma2_rn(a, both(0.36f), both(1.0f));
  const float2 t = make_float2(fast_rcp(d.x), fast_rcp(d.y));
  float2 q = __ffma2_rn(t, both(0.047056064f), both(-0.179763913f));
  q = __ffma2_rn(q, t, both(0.180952951f));
  q = __ffma2_rn(q, t, both(0.0265500173f));
  q = __ffma2_rn(q, t, both(0.139719039f));
  q = __ffma2_rn(q, t, both(0.141772494f));
  q = __ffma2_rn(q, t, both(0.143713042f));
  const float2 e = __fmul2_rn(__fmul2_rn(a, a), both(-0.5f * 1.44269504f));
  const float2 phi = __fmul2_rn(__fmul2_rn(q, t), make_float2(fast_ex2(e.x), fast_ex2(e.y)));
  return __ffma2_rn(make_float2(-a.x, -a.y), phi, make_float2(max_nan(x.x, 0.0f), max_nan(x.y, 0.0f)));
}

template <int ACT>
__device__ __forceinline__ float2 act2(float2 x) {
  if (ACT == kActRelu) return make_float2(max_nan(x.x, 0.0f), max_nan(x.y, 0.0f));
  if (ACT == kActSilu) return times_sigmoid2(x, x);
  if (ACT == kActGelu) return gelu2(x);
  if (ACT == kActGeluTanh) {
    const float2 c = __ffma2_rn(__fmul2_rn(x, x), make_float2(0.0713548163f, 0.0713548163f),
                                make_float2(1.59576912f, 1.59576912f));      // 2 sqrt(2/pi) (0.044715 x^2 + 1)
    return times_sigmoid2(x, __fmul2_rn(c, x));
  }
  return x;
}

template <int ACT, int N>
__device__ __forceinline__ void act_each(float (&x)[N]) {
#pragma unroll
  for (int i = 0; i + 1 < N; i += 2) {
    const float2 y = act2<ACT>(make_float2(x[i], x[i + 1]));
    x[i] = y.x, x[i + 1] = y.y;
  }
}

// act over N values (N even), the choice made once.
template <int N>
__device__ __forceinline__ void apply_act_n(float (&x)[N], int act) {
  switch (act) {
    case kActRelu: act_each<kActRelu>(x); break;
    case kActSilu: act_each<kActSilu>(x); break;
    case kActGelu: act_each<kActGelu>(x); break;
    case kActGeluTanh: act_each<kActGeluTanh>(x); break;
    default: break;
  }
}

// x plus 8 residual values (bf16, zeros when there are none), rounded to bf16.
__device__ __forceinline__ uint4 add_round8(const float* x, const uint4& res) {
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

// bias[n .. n+7] (n % 8 == 0), or zeros.
__device__ __forceinline__ void load_bias8(const EpiArgs& e, uint64_t n, float (&b)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) b[i] = 0.0f;
  if (e.bias == nullptr) return;
  if (e.bias_f32) {
    const float4* v = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(e.bias) + n);
    const float4 b0 = __ldg(v), b1 = __ldg(v + 1);
    b[0] = b0.x, b[1] = b0.y, b[2] = b0.z, b[3] = b0.w;
    b[4] = b1.x, b[5] = b1.y, b[6] = b1.z, b[7] = b1.w;
  } else {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(e.bias) + n));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      b[2 * i] = __uint_as_float(w[i] << 16);
      b[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}

// The epilogue of a warp's 32 rows x P * 32 columns, 32 columns a pass through
// the warp's shared-memory slot (4 KB).  put(p, at) writes the pass's 32
// accumulators of the lane's row: 16-byte chunk c to at(c).  Read back, four
// neighbouring lanes hold a row's 32 columns, eight each, so that the
// residual's loads and the output's stores are whole sectors, and a lane works
// on four rows at once.  The loop over the passes stays rolled: unrolled over
// 128 columns the arithmetic was code that no instruction cache kept (4096^3
// with bias, gelu and residual: 163 us, where the plain GEMM takes 80).
//   m0, n0   the first row and column; rows >= row_end are not stored.
template <int P, typename Put>
__device__ __forceinline__ void staged_epilogue(const Put& put, uint8_t* slot, int lane, const EpiArgs& e,
                                                __nv_bfloat16* Y, int N, int m0, int row_end, int n0) {
  const int q = lane & 3, r0 = lane >> 2;    // columns 8 q .. 8 q + 7 of rows r0 + 8 i
  auto chunk = [&](int r, int c) { return reinterpret_cast<float4*>(slot + r * 128 + ((c ^ (r & 7)) << 4)); };
#pragma unroll 1
  for (int p = 0; p < P; ++p) {
    const int n = n0 + p * 32 + q * 8;
    uint4 res[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) res[i] = make_uint4(0, 0, 0, 0);
    if (e.residual != nullptr) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int m = m0 + r0 + 8 * i;
        if (m < row_end) res[i] = *reinterpret_cast<const uint4*>(e.residual + static_cast<uint64_t>(m) * e.ld_r + n);
      }
    }
    float b[8];
    load_bias8(e, n, b);
    put(p, [&](int c) { return chunk(lane, c); });
    __syncwarp();
    float x[32];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 v = *chunk(r0 + 8 * i, 2 * q + h);
        x[8 * i + 4 * h + 0] = v.x + b[4 * h + 0];
        x[8 * i + 4 * h + 1] = v.y + b[4 * h + 1];
        x[8 * i + 4 * h + 2] = v.z + b[4 * h + 2];
        x[8 * i + 4 * h + 3] = v.w + b[4 * h + 3];
      }
    }
    __syncwarp();                            // the slot may be written again
    apply_act_n(x, e.act);
    FGFP8_DCHECK(n + 8 <= N);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = m0 + r0 + 8 * i;
      if (m < row_end) *reinterpret_cast<uint4*>(Y + static_cast<uint64_t>(m) * N + n) = add_round8(x + 8 * i, res[i]);
    }
  }
}

// The same for a warp whose lanes have 128 columns each of their own row in
// registers (accumulators as fp32 bits), with a smaller slot (2 KB): the
// arithmetic stays with the row's lane, and the residual and the output pass
// through the slot as bf16, 32 columns a step, so that four neighbouring lanes
// move 64 bytes of a row.  Lanes that read and wrote their own rows, 16 bytes
// at a time, held up the next tile's operands in the same memory (4096 x 14336
// x 4096: with a residual 231 us, through the slot 204; bias, gelu and residual
// 235 and 216, 222 with gelu's present fit; none of them 200 and 194).  The residual alone through the slot
// left half of that, and reading it a step ahead spilled registers.
__device__ __forceinline__ void row_epilogue(const uint32_t (&acc)[128], uint8_t* slot, int lane, const EpiArgs& e,
                                             __nv_bfloat16* Y, int N, int m0, int row_end, int n0) {
  const int q = lane & 3, r0 = lane >> 2;    // 16-byte chunk q of rows r0 + 8 i
  auto chunk = [&](int r, int c) { return reinterpret_cast<uint4*>(slot + r * 64 + ((c ^ ((r >> 1) & 3)) << 4)); };
#pragma unroll
  for (int j = 0; j < 128; j += 32) {
    uint4 own[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) own[i] = make_uint4(0, 0, 0, 0);
    if (e.residual != nullptr) {
      uint4 res[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int m = m0 + r0 + 8 * i;
        res[i] = make_uint4(0, 0, 0, 0);
        if (m < row_end)
          res[i] = *reinterpret_cast<const uint4*>(e.residual + static_cast<uint64_t>(m) * e.ld_r + n0 + j + 8 * q);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) *chunk(r0 + 8 * i, q) = res[i];
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 4; ++i) own[i] = *chunk(lane, i);
      __syncwarp();
    }
    float x[32];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float b[8];
      load_bias8(e, n0 + j + 8 * i, b);
#pragma unroll
      for (int k = 0; k < 8; ++k) x[8 * i + k] = __uint_as_float(acc[j + 8 * i + k]) + b[k];
    }
    apply_act_n(x, e.act);
#pragma unroll
    for (int i = 0; i < 4; ++i) *chunk(lane, i) = add_round8(x + 8 * i, own[i]);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = m0 + r0 + 8 * i;
      const uint4 v = *chunk(r0 + 8 * i, q);
      if (m < row_end) *reinterpret_cast<uint4*>(Y + static_cast<uint64_t>(m) * N + n0 + j + 8 * q) = v;
    }
    __syncwarp();                            // the slot may be written again
  }
}

__device__ __forceinline__ float load_bias(const EpiArgs& e, uint64_t n) {
  if (e.bias == nullptr) return 0.0f;
  return e.bias_f32 ? __ldg(reinterpret_cast<const float*>(e.bias) + n)
                    : __bfloat162float(__ldg(reinterpret_cast<const __nv_bfloat16*>(e.bias) + n));
}

}  // namespace fgfp8
