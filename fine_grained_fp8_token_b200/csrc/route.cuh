// Router of an expert layer: the scores of E experts -> each token's topk
// experts and their weights.
//
//   softmax  key_e = z_e                      p_e = exp(z_e - max z) / sum_e exp(z_e - max z)
//   sigmoid  key_e = sigma(z_e) + bias_e      p_e = sigma(z_e)
//
// An expert whose key is -inf or NaN is never chosen.  With groups, the experts
// form n_group equal runs; a group's score is its largest key (softmax) or the
// sum of its two largest (sigmoid), and only the topk_group best groups
// compete.  The topk largest keys are chosen in descending order, ties to the
// lowest index; w_j = p_j, divided by the chosen p's sum when renormalized,
// times the factor.  Slots that find no expert get id -1 and weight 0.
#pragma once
#include <cuda_bf16.h>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "ptx.cuh"

namespace fgfp8 {

struct RouteArgs {
  const void* logits;
  uint64_t ld;
  const float* bias;
  int T, E, topk, n_group, topk_group, renormalize;
  float scale;
  int32_t* ids;
  float* weights;
};

constexpr int kRouteWarps = 4;                // tokens per CTA

__device__ __forceinline__ float load_logit(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load_logit(const __nv_bfloat16* p) { return __bfloat162float(__ldg(p)); }

// One warp per token; lane l holds the experts l, l + 32, ....
template <int EPL, bool kSigmoid, typename In>
__global__ void __launch_bounds__(kRouteWarps * 32) route_topk_kernel(const RouteArgs p) {
  using Key = typename std::conditional<kSigmoid, double, float>::type;
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
  if (t >= p.T) return;
  const Key kNone = static_cast<Key>(-INFINITY);
  const In* row = reinterpret_cast<const In*>(p.logits) + static_cast<uint64_t>(t) * p.ld;

  float z[EPL];
  Key key[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 32 * i;
    z[i] = e < p.E ? load_logit(row + e) : -INFINITY;
    if (!(z[i] > -INFINITY)) z[i] = -INFINITY;                    // NaN too
    if constexpr (kSigmoid) {
      key[i] = kNone;
      if (z[i] > -INFINITY) {
        const double b = p.bias != nullptr ? static_cast<double>(__ldg(p.bias + e)) : 0.0;
        key[i] = 1.0 / (1.0 + exp(-static_cast<double>(z[i]))) + b;
        if (!(key[i] > kNone)) key[i] = kNone;
      }
    } else {
      key[i] = z[i];
    }
  }

  if (p.n_group > 1) {
    const int per = p.E / p.n_group;
    Key score = kNone;                                            // lane g: the score of group g
    for (int g = 0; g < p.n_group; ++g) {
      Key a = kNone, b = kNone;                                   // the two largest
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int e = lane + 32 * i;
        if (e / per == g && e < p.E) {
          if (key[i] > a) b = a, a = key[i];
          else if (key[i] > b) b = key[i];
        }
      }
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const Key a2 = __shfl_xor_sync(0xFFFFFFFFu, a, d), b2 = __shfl_xor_sync(0xFFFFFFFFu, b, d);
        const Key lo = a2 > a ? a : a2;
        a = a2 > a ? a2 : a;
        b = b2 > b ? b2 : b;
        b = lo > b ? lo : b;
      }
      if (lane == g) score = (kSigmoid && b > kNone) ? a + b : a;
    }
    // rank of each group: better groups, and equal ones of lower index
    int before = 0;
    for (int g = 0; g < p.n_group; ++g) {
      const Key o = __shfl_sync(0xFFFFFFFFu, score, g);
      before += (o > score || (o == score && g < lane)) ? 1 : 0;
    }
    const uint32_t kept = __ballot_sync(0xFFFFFFFFu, lane < p.n_group && before < p.topk_group);
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + 32 * i;
      if (e < p.E && !((kept >> (e / per)) & 1u)) key[i] = kNone;
    }
  }

  float zmax = -INFINITY, sum = 0.0f;
  if constexpr (!kSigmoid) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) zmax = fmaxf(zmax, z[i]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) zmax = fmaxf(zmax, __shfl_xor_sync(0xFFFFFFFFu, zmax, d));
  }
  // a logit of +inf takes the whole softmax (shared by all such logits)
  auto weight_of = [&](float x) -> float {
    if constexpr (kSigmoid) return __fdiv_rn(1.0f, 1.0f + expf(-x));
    if (x == -INFINITY) return 0.0f;
    return x == zmax ? 1.0f : expf(x - zmax);
  };
  if constexpr (!kSigmoid) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) sum += weight_of(z[i]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
  }

  int my_id = -1;
  float my_w = 0.0f;
  for (int j = 0; j < p.topk; ++j) {
    Key best = kNone;
    int at = 0x7FFFFFFF;
    float zb = 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (key[i] > best) best = key[i], at = lane + 32 * i, zb = z[i];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      const Key ob = __shfl_xor_sync(0xFFFFFFFFu, best, d);
      const int oa = __shfl_xor_sync(0xFFFFFFFFu, at, d);
      const float oz = __shfl_xor_sync(0xFFFFFFFFu, zb, d);
      if (ob > best || (ob == best && oa < at)) best = ob, at = oa, zb = oz;
    }
    if (!(best > kNone)) break;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (lane + 32 * i == at) key[i] = kNone;
    if (lane == j) my_id = at, my_w = weight_of(zb);
  }

  float total = sum;
  if (p.renormalize) {
    total = my_w;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, d);
    total = fmaxf(total, 1e-20f);
  } else if (kSigmoid) {
    total = 1.0f;
  }
  if (lane < p.topk) {
    p.ids[static_cast<uint64_t>(t) * p.topk + lane] = my_id;
    p.weights[static_cast<uint64_t>(t) * p.topk + lane] = my_id < 0 ? 0.0f : __fdiv_rn(my_w, total) * p.scale;
  }
}

}  // namespace fgfp8
