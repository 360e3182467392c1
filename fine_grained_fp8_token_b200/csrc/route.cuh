// Router of an expert layer: the scores of E experts -> each token's topk
// experts and their weights.
//
//   softmax  key_e = z_e                      p_e = exp(z_e - max z) / sum_e exp(z_e - max z)
//   sigmoid  key_e = sigma(z_e) + bias_e      p_e = sigma(z_e)
//
// (Without a bias sigmoid keys order as the logits do, and z_e is compared.)
// An expert whose key is -inf or NaN is never chosen.  With groups, the experts
// form n_group equal runs; a group's score is its largest key (softmax) or the
// sum of its two largest sigma(z) + bias (sigmoid), and only the topk_group
// best groups compete.  The topk largest keys are chosen in descending order,
// ties to the lowest index; w_j = p_j, divided by the chosen p's sum when
// renormalized, times the factor.  Slots that find no expert get id -1 and
// weight 0.
//
// One warp per token: lane l holds EPL consecutive experts as order-preserving
// integers, sorted once in registers.  A round of the selection is then one
// warp-wide redux over the lanes' heads and a ballot, whose lowest lane is the
// lowest index; the winner drops its head.  Which of its experts that was is
// found for all slots together at the end.  The kernel is bound by issuing
// instructions, not by its 4 E bytes per token.  Counted with 8 experts a lane,
// per token: 30 a round, and around the rounds 300 (fp32 softmax) to 360 (bf16),
// 570 with biased sigmoids and 940 with groups on top (the keys staged in shared
// memory and scanned).  20011 tokens x 160 softmax, 6 of them, are 545 x 20011 =
// 10.9 M, 9.4 us of the SMs' issue slots at 1.965 GHz, and take 11.5 us; 8192 x
// 256 in 8 groups with a bias 1200 x 8192 = 9.8 M and 16 us; one token 3.7 us
// (selecting with a lane's maximum and 64-bit shuffles took 49, 27 and 14 us for
// the second, the first and the last).
//
// sigma(z) + bias is defined in 64 bits.  The warp forms it in 32 and looks at
// the gaps its decisions rest on; where one is within the 32-bit error, it
// keeps choosing until a gap is clear and orders the chosen in 64 bits, a lane
// each (groups: all keys in 64 bits, exact_groups).  Forming every key of every
// token in 64 bits cost 50 us for 8192 tokens x 256 experts.
#pragma once
#include <cuda_bf16.h>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "ptx.cuh"
#include "quant.cuh"

namespace fgfp8 {

struct RouteArgs {
  const void* logits;
  uint64_t ld;
  const float* bias;
  int T, E, topk, n_group, topk_group, renormalize;
  int vec;                                    // rows allow 16-byte loads
  int group_lanes;                            // log2 of the lanes that scan a group
  FastDiv per{1};                             // experts per group
  float scale;
  int32_t* ids;
  float* weights;
};

constexpr int kRouteWarps = 4;                // tokens per CTA
constexpr int kRouteMaxExperts = 512;

// Order-preserving integer of an fp32 number (the two zeros alike); -inf and
// NaN map to 0, below every other number's.
__device__ __forceinline__ uint32_t order_of(float x) {
  if (!(x > -INFINITY)) return 0u;
  const uint32_t b = __float_as_uint(__fadd_rn(x, 0.0f));
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return o == 0u ? -INFINITY : __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}

// From exp(-|z|), which keeps results below fp32's normal numbers and does not overflow.
__device__ __forceinline__ float sigmoid_f32(float z) {
  const float e = expf(-fabsf(z));
  return __fdiv_rn(z < 0.0f ? e : 1.0f, 1.0f + e);
}

// sigma(z) for the 32-bit keys, from the hardware's exponential and division.
// With r the relative error of exp(-z), 2^-22 + |z| 2^-24, sigma is off by
// sigma (1 - sigma) r <= 2^-24 + 0.23 2^-24, and by 2 ulp of the division:
// less than 2^-21.  The sum with the bias is rounded once more, 2^-24 |k|.
__device__ __forceinline__ float sigmoid_key(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }
__device__ __forceinline__ float key_slack(float k) { return 9.5367432e-7f * fmaxf(1.0f, fabsf(k)); }   // 2^-20

template <int EPL, typename In>
__device__ __forceinline__ void load_logits(const RouteArgs& p, const In* row, int lane, float (&z)[EPL]) {
  const int e0 = lane * EPL;
  constexpr int kPer16 = 16 / sizeof(In);
  if constexpr (EPL * sizeof(In) >= 16) {
    if (p.vec && e0 + EPL <= p.E) {
#pragma unroll
      for (int c = 0; c < EPL / kPer16; ++c) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(row + e0) + c);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (sizeof(In) == 4) {
            z[c * 4 + i] = __uint_as_float(w[i]);
          } else {
            z[c * 8 + 2 * i] = __uint_as_float(w[i] << 16);
            z[c * 8 + 2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
          }
        }
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    z[i] = -INFINITY;
    if (e0 + i < p.E) {
      if constexpr (sizeof(In) == 4) z[i] = __ldg(row + e0 + i);
      else z[i] = __bfloat162float(__ldg(row + e0 + i));
    }
  }
}

// Lane g < n_group: the two largest of the group's keys[E] (shared memory;
// `none` below all of them), 2^group_lanes lanes per group.
template <typename Key>
__device__ __forceinline__ void group_top2(const Key* keys, const RouteArgs& p, int lane, Key none, Key& first,
                                           Key& second) {
  const int lanes = 1 << p.group_lanes, per = p.per.d;
  const int g = lane >> p.group_lanes, s = lane & (lanes - 1);
  const int count = g < p.n_group && s < per ? (per - s + lanes - 1) >> p.group_lanes : 0;
  int r = g < count ? g : 0;                  // groups start apart, so their reads fall into different banks
  Key a = none, b = none;
  for (int j = 0; j < count; ++j) {
    const Key k = keys[g * per + s + (r << p.group_lanes)];
    if (++r == count) r = 0;
    const Key lo = k > a ? a : k;
    a = k > a ? k : a;
    b = lo > b ? lo : b;
  }
#pragma unroll 1
  for (int d = 1; d < lanes; d <<= 1) {
    const Key a2 = __shfl_xor_sync(0xFFFFFFFFu, a, d), b2 = __shfl_xor_sync(0xFFFFFFFFu, b, d);
    const Key lo = a2 > a ? a : a2;
    a = a2 > a ? a2 : a;
    b = b2 > b ? b2 : b;
    b = lo > b ? lo : b;
  }
  first = __shfl_sync(0xFFFFFFFFu, a, (lane << p.group_lanes) & 31);
  second = __shfl_sync(0xFFFFFFFFu, b, (lane << p.group_lanes) & 31);
}

// Groups that compete, a bit each: lane g holds group g's score.
template <typename Key>
__device__ __forceinline__ uint32_t best_groups(Key score, const RouteArgs& p, int lane) {
  int before = 0;
  for (int g = 0; g < p.n_group; ++g) {
    const Key o = __shfl_sync(0xFFFFFFFFu, score, g);
    before += (o > score || (o == score && g < lane)) ? 1 : 0;
  }
  return __ballot_sync(0xFFFFFFFFu, lane < p.n_group && before < p.topk_group);
}

// sigma(z) in 64 bits: exp(-z) by Cody and Waite's reduction, x = n ln 2 + r
// with ln 2 as a 40-bit head (n * head is exact) and a tail, and the Taylor
// series of e^r to r^13 (|r| <= 0.35: below 2^-57).  |z| is cut at 708, where
// sigma is 1 or below 2^-1021.
__device__ __forceinline__ double sigmoid_f64(float z) {
  const double x = fmin(fmax(-static_cast<double>(z), -708.0), 708.0);
  const double n = rint(x * 1.4426950408889634);
  const double r = __fma_rn(-n, -1.7239444525614835e-13, __fma_rn(-n, 0.6931471805601177, x));
  double e = 1.0 / 6227020800.0;
  e = __fma_rn(e, r, 1.0 / 479001600.0);
  e = __fma_rn(e, r, 1.0 / 39916800.0);
  e = __fma_rn(e, r, 1.0 / 3628800.0);
  e = __fma_rn(e, r, 1.0 / 362880.0);
  e = __fma_rn(e, r, 1.0 / 40320.0);
  e = __fma_rn(e, r, 1.0 / 5040.0);
  e = __fma_rn(e, r, 1.0 / 720.0);
  e = __fma_rn(e, r, 1.0 / 120.0);
  e = __fma_rn(e, r, 1.0 / 24.0);
  e = __fma_rn(e, r, 1.0 / 6.0);
  e = __fma_rn(e, r, 0.5);
  e = __fma_rn(e, r, 1.0);
  e = __fma_rn(e, r, 1.0);
  const double two_n = __hiloint2double((1023 + static_cast<int>(n)) << 20, 0);
  return __drcp_rn(__fma_rn(e, two_n, 1.0));
}

// The 64-bit keys of this lane's experts into keys[]; the loops of this rare
// path stay rolled and in shared memory, so that it costs the common one no
// registers.
template <int EPL, typename In>
__device__ __forceinline__ void exact_keys(const RouteArgs& p, const In* row, uint32_t kept, double* keys) {
  const int e0 = (threadIdx.x & 31) * EPL;
  __syncwarp();                               // the 32-bit keys in this memory have been read
#pragma unroll 1
  for (int e = e0; e < e0 + EPL; ++e) {
    double k = static_cast<double>(-INFINITY);
    if (e < p.E && ((kept >> (p.per.div(e) & 31)) & 1u)) {
      const float z = static_cast<float>(row[e]);
      if (z > -INFINITY) k = sigmoid_f64(z) + (p.bias != nullptr ? __ldg(p.bias + e) : 0.0f);
      if (!(k > static_cast<double>(-INFINITY))) k = static_cast<double>(-INFINITY);
    }
    keys[e] = k;
  }
  __syncwarp();
}

// The groups that compete, decided in 64 bits.
template <int EPL, typename In>
__device__ __forceinline__ uint32_t exact_groups(const RouteArgs& p, const In* row, double* keys) {
  const int lane = threadIdx.x & 31;
  exact_keys<EPL>(p, row, 0xFFFFFFFFu, keys);
  double a, b;
  group_top2(keys, p, lane, static_cast<double>(-INFINITY), a, b);
  return best_groups(b > static_cast<double>(-INFINITY) ? a + b : a, p, lane);
}

// The choice in 64 bits among all experts of the kept groups, for tokens with
// more close keys than lanes: the expert of slot j in sel[j]; returns how many.
template <int EPL, typename In>
__device__ __forceinline__ int exact_choice(const RouteArgs& p, const In* row, uint32_t kept, double* keys, int* sel) {
  const int lane = threadIdx.x & 31, e0 = lane * EPL;
  const double kNone = static_cast<double>(-INFINITY);
  exact_keys<EPL>(p, row, kept, keys);
  int found = 0;
#pragma unroll 1
  for (; found < p.topk; ++found) {
    double best = kNone;
    int at = e0;
#pragma unroll 1
    for (int e = e0; e < e0 + EPL; ++e)
      if (keys[e] > best) best = keys[e], at = e;
#pragma unroll 1
    for (int d = 16; d > 0; d >>= 1) {
      const double ob = __shfl_xor_sync(0xFFFFFFFFu, best, d);
      const int oa = __shfl_xor_sync(0xFFFFFFFFu, at, d);
      if (ob > best || (ob == best && oa < at)) best = ob, at = oa;
    }
    if (!(best > kNone)) break;
    if (at / EPL == lane) {
      keys[at] = kNone;
      sel[found] = at;
    }
  }
  __syncwarp();
  return found;
}

// Batcher's odd-even merge sort of N = 2^k registers, descending.
template <int N>
__device__ __forceinline__ void sort_descending(uint32_t (&k)[N]) {
#pragma unroll
  for (int p = 1; p < N; p <<= 1)
#pragma unroll
    for (int q = p; q > 0; q >>= 1)
#pragma unroll
      for (int j = q % p; j + q < N; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i)
          if (j + i + q < N && (j + i) / (2 * p) == (j + i + q) / (2 * p)) {
            const uint32_t a = k[j + i], b = k[j + i + q];
            k[j + i] = max(a, b);
            k[j + i + q] = min(a, b);
          }
}

template <int EPL, bool kSigmoid, typename In>
__global__ void __launch_bounds__(kRouteWarps * 32) route_topk_kernel(const RouteArgs p) {
  __shared__ double s_keys[kRouteWarps][kSigmoid ? EPL * 32 : EPL * 16];   // EPL * 32 integers, or 64-bit keys
  __shared__ int s_sel[kRouteWarps][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int t = blockIdx.x * kRouteWarps + w;
  griddep_launch_dependents();
  griddep_wait();                             // the scores may be the preceding grid's
  if (t >= p.T) return;
  const In* row = reinterpret_cast<const In*>(p.logits) + static_cast<uint64_t>(t) * p.ld;
  const int e0 = lane * EPL;
  const bool biased = kSigmoid && p.bias != nullptr;
  uint32_t* keys = reinterpret_cast<uint32_t*>(s_keys[w]);

  float z[EPL];
  load_logits<EPL>(p, row, lane, z);
  float bias[EPL];
  if (biased) load_logits<EPL>(p, p.bias, lane, bias);
  uint32_t key[EPL];                                              // 0: cannot be chosen
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    if (!(z[i] > -INFINITY)) z[i] = -INFINITY;                    // NaN too
    key[i] = order_of(z[i]);
    if (biased && key[i] != 0u) key[i] = order_of(sigmoid_key(z[i]) + bias[i]);
  }

  uint32_t kept = 0xFFFFFFFFu;
  if (p.n_group > 1) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) keys[e0 + i] = key[i];
    __syncwarp();
    uint32_t first, second;
    group_top2(keys, p, lane, 0u, first, second);
    const float a = value_of(first), b = value_of(second);
    float score = a, slack = 0.0f;
    if (kSigmoid && first != 0u) {
      score = biased ? a : sigmoid_key(a);
      slack = key_slack(score);
      if (second != 0u) {
        const float k = biased ? b : sigmoid_key(b);
        // the keys' slacks, as the two may cancel; twice the keys' errors, they
        // leave room for the rounding of the sum and of score -+ slack
        slack += key_slack(k);
        score += k;
      }
    }
    kept = best_groups(score, p, lane);
    if constexpr (kSigmoid) {
      // the worst group that competes at its lowest against the best that does
      // not at its highest; an infinite or NaN bound is not clear
      const bool in = (kept >> lane) & 1u;
      const uint32_t lo = ~__reduce_max_sync(0xFFFFFFFFu, in ? ~order_of(score - slack) : 0u);
      const uint32_t hi = __reduce_max_sync(0xFFFFFFFFu, !in && lane < p.n_group ? order_of(score + slack) : 0u);
      if (hi != 0u && !(value_of(lo) > value_of(hi))) kept = exact_groups<EPL>(p, row, s_keys[w]);
    }
    const int per = p.per.d;
    int g = p.per.div(e0), left = (g + 1) * per - e0;             // experts left in this lane's group
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      if (left == 0) ++g, left = per;
      --left;
      if (!((kept >> (g & 31)) & 1u)) key[i] = 0u;
    }
    __syncwarp();                                                 // everyone has read the groups' keys
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) keys[e0 + i] = key[i];
  sort_descending<EPL>(key);

  // Rounds: lane j notes the key and the lane of choice j.
  int found = 0;
  uint32_t top_j = 0u;
  int win_j = 0;
  auto choose = [&]() -> bool {
    const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, key[0]);
    if (top == 0u) return false;
    const int win = __ffs(__ballot_sync(0xFFFFFFFFu, key[0] == top)) - 1;
    if (lane == found) top_j = top, win_j = win;
    if (lane == win) {
#pragma unroll
      for (int i = 0; i + 1 < EPL; ++i) key[i] = key[i + 1];
      key[EPL - 1] = 0u;
    }
    ++found;
    return true;
  };
  // biased keys: one more, for the gap behind the last slot
  const int rounds = biased ? p.topk + 1 : p.topk;
  while (found < rounds && choose()) {}
  bool unsure = false, many = false;
  if (biased) {
    // gap between choice j and j + 1, and rounds past it while the last is not clear
    auto unclear_after = [&] {
      const float k = value_of(top_j), next = __shfl_down_sync(0xFFFFFFFFu, k, 1);
      return __ballot_sync(0xFFFFFFFFu, lane + 1 < found && !(k - next > key_slack(k) + key_slack(next)));
    };
    uint32_t unclear = unclear_after();
    unsure = unclear != 0u;
    if (unsure)
      while (found > p.topk && ((unclear >> (found - 2)) & 1u)) {
        many = found == 32;
        if (many || !choose()) break;
        unclear = unclear_after();
      }
  }
  __syncwarp();

  // The expert of choice j: the d-th of lane win_j's keys that equals top_j,
  // d = how many of the choices just before were the same lane's equal keys.
  int e_j = -1;
  {
    int d = 0;
    if (EPL > 1) {
      uint32_t up_top = __shfl_up_sync(0xFFFFFFFFu, top_j, 1);
      int up_win = __shfl_up_sync(0xFFFFFFFFu, win_j, 1);
      bool same = lane > 0 && lane < found && up_top == top_j && up_win == win_j;
      uint32_t run = __ballot_sync(0xFFFFFFFFu, same);
      if (run != 0u) d = __clz(~(run << (31 - lane)));            // ones ending at this lane's bit
    }
    if (lane < found) {
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (keys[win_j * EPL + i] == top_j && d-- == 0) e_j = win_j * EPL + i;
    }
  }
  if constexpr (kSigmoid) {
    if (unsure) {                                                 // the same in every lane
      // order the choices by their keys in 64 bits
      double k = 0.0;
      if (lane < found) {
        k = sigmoid_f64(static_cast<float>(row[e_j])) + __ldg(p.bias + e_j);
      }
      int before = 0;
      for (int o = 0; o < found; ++o) {
        const double ko = __shfl_sync(0xFFFFFFFFu, k, o);
        const int eo = __shfl_sync(0xFFFFFFFFu, e_j, o);
        before += (ko > k || (ko == k && eo < e_j)) ? 1 : 0;
      }
      int* sel = s_sel[w];
      if (many) found = exact_choice<EPL>(p, row, kept, s_keys[w], sel);
      else if (lane < found) sel[before] = e_j;
      __syncwarp();
      if (lane < found) e_j = sel[lane];
    }
  }
  const bool slot = lane < found && lane < p.topk;

  // Weights: lane j has slot j.  The first choice has the largest logit of all
  // (softmax keys are the logits); a logit of +inf takes the whole softmax,
  // shared by all such logits.
  float zj = -INFINITY;
  if (slot) zj = biased ? static_cast<float>(row[e_j]) : value_of(top_j);
  const float zmax = __shfl_sync(0xFFFFFFFFu, zj, 0);
  auto weight_of = [&](float x) -> float {
    if constexpr (kSigmoid) return sigmoid_f32(x);
    if (x == -INFINITY) return 0.0f;
    return x == zmax ? 1.0f : expf(x - zmax);
  };
  const float wt = slot ? weight_of(zj) : 0.0f;
  float total = 1.0f;
  if (p.renormalize) {
    total = wt;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, d);
    total = fmaxf(total, 1e-20f);
  } else if constexpr (!kSigmoid) {
    total = 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) total += weight_of(z[i]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, d);
  }
  if (lane < p.topk) {
    const uint64_t at = static_cast<uint64_t>(t) * p.topk + lane;
    p.ids[at] = slot ? e_j : -1;
    p.weights[at] = slot ? __fdiv_rn(wt, total) * p.scale : 0.0f;
  }
}

}  // namespace fgfp8
