// Few-token kernels (at most 64 tokens): the expert layer's two kernels and
// the linear layer with its epilogue.  All of them read each weight byte once
// and are bound by that read, so one skeleton serves the three:
//
//   kFewGateUp  H[p, :] = quant( silu(g) * u ),  (g, u) = W13[e] quant(x_t)
//   kFewDown    y_t = r_t + sum_e w(t, e) W2[e] H[p, :]
//   kFewLinear  y_m = act(W quant(x_m) + bias) + r_m
//
// (p numbers the pairs of an expert e and a token t routed to it.)  Operands
// are swapped: 128 weight rows are the MMA's M, the tokens its N (16 to 64
// columns), so an expert's few tokens waste no weight bandwidth.  Roles of
// the CTA's warps:
//   promotion   (4 or 8 warps) thread = weight row; per 128-wide K block the
//               partial of each token from TMEM times sa * sw into fp32
//               accumulators, then the epilogue;
//   tokens      (4 warps) each K block belongs to one of them in turn: from bf16 rows it gathers the
//               expert's token rows, quantizes them and writes the 128-byte-
//               swizzled tile; in both cases it writes the products sa * sw.
//               The rows are L2-resident, and quantizing them again per weight
//               block costs a few instructions per 16 KB of weights, which
//               saves a quantizer kernel and the gather of rows.  One warp per
//               block, so that four blocks' loads overlap: the proxy fence
//               before a block is handed over waits for all of its thread's
//               loads (measured with all four warps on every block: 87 us
//               for M = 37, N = 18432, K = 7168);
//   TMA         (1 warp) the weight tiles and, where the source is codes, the
//               token rows (a linear layer's rows are contiguous, and an
//               expert's rows of H are);
//   MMA         (1 warp) owns TMEM, issues the MMAs.
//
// Few rows leave fewer 128-row weight blocks than SMs, so K is split over the
// CTAs of a cluster.  Their partial sums meet in distributed shared memory:
// each rank owns every S-th token, the others store their partials into its
// buffer, and it adds them in rank order.  No global workspace, counters or
// atomics, and the result does not depend on timing.
//
// Every wait is bounded as in the GEMM kernels: on expiry the role records a
// status and unwinds.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cstdint>
#include <type_traits>

#include "epilogue.cuh"
#include "ptx.cuh"
#include "quant.cuh"

namespace fgfp8 {

enum : int { kFewGateUp = 0, kFewDown = 1, kFewLinear = 2 };

constexpr int kFewMaxTokens = 64;
constexpr int kFewMaxExperts = 512;
constexpr int kFewMaxTopk = 16;

struct FewArgs {
  const void* src;                  // token operand: bf16 rows (ld_src in elements) or E4M3 codes (bytes)
  uint64_t ld_src;
  const void* src_scale;            // codes only: Down fp32 [pair, KB], Linear MN-major [KB, ld_s] in `fmt`
  uint64_t ld_s;
  const void* Ws;                   // weight block scales in `fmt`
  int fmt;
  int T;                            // tokens
  int KB;                           // 128-wide K blocks
  int NB;                           // 128-row weight blocks per expert
  const int32_t* ids;               // expert layer: [T, topk]
  const float* wts;                 // expert layer: [T, topk]
  int topk, E;
  uint8_t* Hq;                      // GateUp: codes [pair, I] and scales [pair, I/128]
  float* Hs;
  int I;
  __nv_bfloat16* Y;                 // Down, Linear: [T, N]
  int N;
  EpiArgs epi;
  int lgS;                          // log2 of the cluster size S: ranks that split K
  int early;                        // weights may be requested before the wait for the preceding grid
};

template <int MODE, int NT>
struct FewCfg {
  static constexpr int kTiles = MODE == kFewGateUp ? 2 : 1;          // 128-row weight tiles per stage
  static constexpr uint32_t kABytes = kTiles * 128 * 128;
  static constexpr uint32_t kBBytes = NT * 128;
  static constexpr uint32_t kScBytes = kTiles * NT * 4;
  // tokens per meeting of the ranks, and the largest cluster: its buffer
  // holds max(kRedTok, S) tokens
  static constexpr int kRedTok = MODE == kFewGateUp ? 4 : 8;
  static constexpr int kMaxS = kRedTok;
  // Promotion warpgroups: group g takes the 16-token chunks g, g + 2, ....
  // Two for the wide tile: one group's chain of waits, TMEM loads and FMAs
  // per K block would outlast the 16 KB of weights it covers.
  static constexpr int kGroups = NT == 64 ? 2 : 1;
  static constexpr int kEpiWarps = 4 * kGroups;
  static constexpr int kChunks = NT / 16 / kGroups;                  // chunks per group
  static constexpr uint32_t kRedBytes = kGroups * kRedTok * kTiles * 512;
  static constexpr uint32_t kAccBytes = MODE == kFewDown ? NT * 512 : 0;
  static constexpr int kPairs = NT * kFewMaxTopk;
  static constexpr int kActive = kPairs < kFewMaxExperts ? kPairs : kFewMaxExperts;
  using Mask = typename std::conditional<NT == 64, unsigned long long, unsigned int>::type;   // a bit per token
  static constexpr uint32_t kMaskBytes = MODE == kFewLinear ? 0 : kFewMaxExperts * sizeof(Mask);
  static constexpr uint32_t kListBytes = MODE == kFewLinear ? 0 : kActive * 4;      // expert ids and first pairs, u16
  static constexpr uint32_t kWeightBytes = MODE == kFewDown ? kPairs * 6 : 0;       // fp32 weights, i16 ids
  static constexpr uint32_t kAmaxBytes = MODE == kFewGateUp ? 2 * 4 * NT * 4 : 0;
  static constexpr uint32_t kBarrierBytes = NT == 64 ? 320 : 256;
  // Two CTAs per SM while the token tile is small: one CTA's ramp and
  // epilogue run under the other's stream.
  static constexpr int kCtas = NT == 16 ? 2 : 1;
  static constexpr uint32_t kBudget = (kCtas == 2 ? 115712u : 232448u) - 1024u;     // after the 1 KB alignment
  static constexpr uint32_t kFixed =
      kRedBytes + kAccBytes + kMaskBytes + kListBytes + kWeightBytes + kAmaxBytes + kBarrierBytes;
  static constexpr uint32_t kStageBytes = kABytes + kBBytes + kScBytes;
  static constexpr int kStagesFit = static_cast<int>((kBudget - kFixed) / kStageBytes);
  static constexpr int kStages = kStagesFit > 8 ? 8 : kStagesFit;
  static constexpr size_t kSmemBytes = 1024 + kFixed + static_cast<size_t>(kStages) * kStageBytes;
  // Warps that prepare token operands, K block u by warp u % kTokWarps.  At
  // most kStages: a warp that has passed its wait for block u - kTokWarps
  // knows that block u - kTokWarps - kStages is consumed, and its parity
  // wait for block u tells phases apart only if that covers u - 2 kStages.
  static constexpr int kTokWarps = kStages < 4 ? kStages : 4;
  static constexpr int kNumBuf = MODE == kFewGateUp && NT == 64 ? 2 : 4;             // TMEM partial buffers
  static constexpr uint32_t kBufCols = kTiles * NT;
  static constexpr uint32_t kTmemCols = kNumBuf * kBufCols;                          // 64, 128 or 256
  static constexpr int kThreads = (kEpiWarps + 6) * 32;
  static_assert(kStages >= 3, "pipeline depth");
  static_assert(kTokWarps <= kStages && kTokWarps <= 4, "parity waits of the token warps");
  static_assert(kTmemCols >= 32 && (kTmemCols & (kTmemCols - 1)) == 0 && kTmemCols * kCtas <= 512, "TMEM columns");
  static_assert((2 * kStages + 2 * kNumBuf + 8) * 8 + 16 <= kBarrierBytes, "barrier area");
};

// ------------------------------------------------------------ cluster helpers
__device__ __forceinline__ uint32_t cluster_ctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t map_to_rank(uint32_t smem_addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return done != 0;
}
// mbar_wait with acquire at cluster scope (arrivals from other CTAs).
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait_cluster(bar, parity)) return true;
  const uint64_t start = globaltimer_ns();
  uint32_t spins = 0;
  while (!mbar_try_wait_cluster(bar, parity)) {
    if ((++spins & 0xFFu) == 0 && globaltimer_ns() - start > kWaitLimitNs) return false;
  }
  return true;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// ------------------------------------------------------------ scales
// fp32 value of a stored scale: fp32 bits, or the power of two of a UE8M0
// byte (0 = 2^-127, 255 = NaN).
__device__ __forceinline__ float scale_value(uint32_t raw, int fmt) {
  if (fmt == 0) return __uint_as_float(raw);
  if (raw == 0u) return __uint_as_float(0x00400000u);
  return raw == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(raw << 23);
}
__device__ __forceinline__ uint32_t load_scale_word(const void* p, uint64_t i, int fmt) {
  return fmt == 0 ? __ldg(reinterpret_cast<const uint32_t*>(p) + i) : __ldg(reinterpret_cast<const uint8_t*>(p) + i);
}

// Scale of a group whose amax is a full fp32 number: max(amax, 1e-4) / 448
// (IEEE division), or the smallest power of two not below that.
__device__ __forceinline__ float scale_of_f32(float amax, int fmt) {
  const float s = __fdiv_rn(amax < 1e-4f ? 1e-4f : amax, 448.0f);
  if (fmt == 0) return s;
  uint32_t b = __float_as_uint(s), e = b >> 23;
  if ((b & 0x7FFFFFu) != 0u && e < 255u) e += 1u;
  return scale_value(e, 1);
}

// Position of the i-th set bit of m (i < popcount).
__device__ __forceinline__ int nth_bit(uint64_t m, int i) {
  for (; i > 0; --i) m &= m - 1;
  return __ffsll(static_cast<long long>(m)) - 1;
}

// ------------------------------------------------------------ work of a CTA
// A segment: K blocks [kb0, kb1) of one expert's weight rows.
struct FewSeg {
  int a, e;                         // position in the active list, expert
  int j;                            // GateUp: 128-wide block of I; else the 128-row block of N
  int kb0, kb1;
};

// The segments of one CTA, the same sequence for every role.
//   GateUp  items (a, j) strided over the clusters, rank r taking its S-th of K
//   Down    the cluster's block of 128 output columns: the (a, kb) blocks of
//           all active experts in one line, cut into S equal ranges
//   Linear  the cluster's block of 128 output columns, rank r its S-th of K
template <int MODE>
struct FewIter {
  int pos, end, step, KB, NJ, j, kb0, kb1;
  const uint16_t* act;
  __device__ FewIter(const FewArgs& p, int active, const uint16_t* act_, int rank, int cluster, int clusters) {
    act = act_;
    KB = p.KB;
    NJ = p.I / 128;
    j = cluster;
    if (MODE == kFewGateUp) {
      pos = cluster, end = active * NJ, step = clusters;
      kb0 = KB * rank >> p.lgS, kb1 = KB * (rank + 1) >> p.lgS;
    } else if (MODE == kFewDown) {
      const int units = active * KB;                  // at most 2^9 experts x 2^13 blocks
      pos = units * rank >> p.lgS;
      end = units * (rank + 1) >> p.lgS;
    } else {
      pos = 0, end = 1;
      kb0 = KB * rank >> p.lgS, kb1 = KB * (rank + 1) >> p.lgS;
    }
  }
  __device__ bool next(FewSeg& s) {
    if (pos >= end) return false;
    if (MODE == kFewGateUp) {
      s.a = pos / NJ;
      s.j = pos - s.a * NJ;
      s.e = act[s.a];
      s.kb0 = kb0, s.kb1 = kb1;
      pos += step;
    } else if (MODE == kFewDown) {
      s.a = pos / KB;
      s.e = act[s.a];
      s.j = j;
      s.kb0 = pos - s.a * KB;
      s.kb1 = s.kb0 + (end - pos) < KB ? s.kb0 + (end - pos) : KB;
      pos += s.kb1 - s.kb0;
    } else {
      s.a = 0, s.e = 0, s.j = j, s.kb0 = kb0, s.kb1 = kb1;
      pos = end;
    }
    return true;
  }
};

template <int MODE, int NT, bool kBf16>
__global__ void __launch_bounds__(FewCfg<MODE, NT>::kThreads, FewCfg<MODE, NT>::kCtas)
    few_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
               const __grid_constant__ FewArgs p) {
  using C = FewCfg<MODE, NT>;
  constexpr bool kMoe = MODE != kFewLinear;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = sA + C::kStages * C::kABytes;
  float* sSc = reinterpret_cast<float*>(sB + C::kStages * C::kBBytes);             // [stage][tile][NT]
  float* sAcc = sSc + C::kStages * C::kTiles * NT;                                 // Down: [token][128]
  float* sRed = sAcc + C::kAccBytes / 4;                                           // [rank][slot][tile][128]
  typename C::Mask* sMask = reinterpret_cast<typename C::Mask*>(sRed + C::kRedBytes / 4);   // tokens of each expert
  float* sWt = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(sMask) + C::kMaskBytes);   // Down: [T * topk]
  float* sAmax = sWt + (MODE == kFewDown ? C::kPairs : 0);                         // GateUp: [2][4][NT]
  uint16_t* sAct = reinterpret_cast<uint16_t*>(sAmax + C::kAmaxBytes / 4);         // active experts
  uint16_t* sBase = sAct + (kMoe ? C::kActive : 0);                                // their first pairs
  int16_t* sIds = reinterpret_cast<int16_t*>(sBase + (kMoe ? C::kActive : 0));     // Down: [T * topk]
  uint64_t* full = reinterpret_cast<uint64_t*>(sIds + (MODE == kFewDown ? C::kPairs : 0));
  uint64_t* empty = full + C::kStages;
  uint64_t* tfull = empty + C::kStages;
  uint64_t* tempty = tfull + C::kNumBuf;
  uint64_t* mma_done = tempty + C::kNumBuf;
  uint64_t* red_full = mma_done + 1;
  uint64_t* red_empty = red_full + 2;
  uint64_t* amax_bar = red_empty + 2;
  uint64_t* seg_bar = amax_bar + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(seg_bar + 1);
  int* s_active = reinterpret_cast<int*>(tmem_slot + 1);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kTokWarp0 = C::kEpiWarps, kTmaWarp = kTokWarp0 + 4, kMmaWarp = kTmaWarp + 1;
  const int lgS = p.lgS, S = 1 << lgS;
  const int rank = S > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int cluster = static_cast<int>(blockIdx.x) >> lgS, clusters = static_cast<int>(gridDim.x) >> lgS;

  if (tid == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1 + 1);                 // the TMA's expect and the block's token warp
      mbar_init(&empty[s], 1 + C::kEpiWarps);     // the MMAs and the promotion warps (scales)
    }
    for (int b = 0; b < C::kNumBuf; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], C::kEpiWarps);
    }
    mbar_init(mma_done, 1);
    for (int g = 0; g < 2; ++g) {
      mbar_init(&red_full[g], 4 * S);
      mbar_init(&red_empty[g], 4 * S);
      mbar_init(&amax_bar[g], 4);
    }
    mbar_init(seg_bar, C::kEpiWarps);
    fence_mbarrier_init();
    tma_prefetch_desc(&tmW);
    if (!kBf16) tma_prefetch_desc(&tmX);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }

  // GateUp reads the routing that the preceding grid may have written, and
  // lets Down start as soon as every CTA here has passed its wait: Down's
  // CTAs then request weights while the last CTAs here finish.  For Down the
  // routing is complete before it starts (GateUp waited for it), so only H
  // and the output wait for GateUp.
  if (MODE == kFewGateUp) {
    griddep_wait();
    griddep_launch_dependents();
  }
  if constexpr (kMoe) {
    const int P = p.T * p.topk;
    for (int e = tid; e < p.E; e += C::kThreads) sMask[e] = 0;
    if constexpr (MODE == kFewDown)
      for (int i = tid; i < NT * 128; i += C::kThreads) sAcc[i] = 0.0f;
    __syncthreads();
    for (int i = tid; i < P; i += C::kThreads) {
      const int id = __ldg(p.ids + i);
      const bool in = id >= 0 && id < p.E;
      if (in) atomicOr(sMask + id, typename C::Mask(1) << (i / p.topk));
      if (id >= p.E && blockIdx.x == 0) record_status(kDevBadExpert);
      if constexpr (MODE == kFewDown) {
        sIds[i] = static_cast<int16_t>(in ? id : -1);
        sWt[i] = __ldg(p.wts + i);
      }
    }
    __syncthreads();
    if (warp == 0) {
      int na = 0, np = 0;
      for (int e0 = 0; e0 < p.E; e0 += 32) {
        const int e = e0 + lane;
        const uint64_t m = e < p.E ? sMask[e] : 0;
        const int c = __popcll(m);
        int incl = c;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
          if (lane >= d) incl += o;
        }
        const uint32_t on = __ballot_sync(0xFFFFFFFFu, c != 0);
        if (c != 0) {
          const int a = na + __popc(on & ((1u << lane) - 1u));
          sAct[a] = static_cast<uint16_t>(e);
          sBase[a] = static_cast<uint16_t>(np + incl - c);
        }
        na += __popc(on);
        np += __shfl_sync(0xFFFFFFFFu, incl, 31);
      }
      if (lane == 0) *s_active = na;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (S > 1) cluster_sync();                      // the ranks' barriers exist before anyone arrives on them
  const uint32_t tmem_base = *tmem_slot;
  const int active = kMoe ? *s_active : 1;
  FewIter<MODE> work(p, active, sAct, rank, cluster, clusters);
  FewSeg sg{};
  // tokens of a segment's expert
  auto tokens_of = [&](const FewSeg& s) -> uint64_t {
    if constexpr (kMoe) return sMask[s.e];
    return p.T >= 64 ? ~0ull : (1ull << p.T) - 1ull;
  };
  const bool weights_early = MODE == kFewDown || (MODE == kFewLinear && p.early);
  if (!(warp == kTmaWarp && weights_early)) griddep_wait();

  if (warp == kTmaWarp) {
    if (lane == 0) {
      // ================= weight tiles, and token tiles of codes
      const FewIter<MODE> from_start = work;
      uint32_t it = 0;
      bool ok = true;
      auto weights = [&](uint32_t u, int kb) {
        const int row = (sg.e * p.NB + (MODE == kFewGateUp ? 2 * sg.j : sg.j)) * 128;
        const int s = u % C::kStages;
        const uint32_t b_bytes = kBf16 ? 0u : static_cast<uint32_t>(((__popcll(tokens_of(sg)) + 15) & ~15) * 128);
        mbar_arrive_expect_tx(&full[s], C::kABytes + b_bytes);
        tma_load_2d(sA + s * C::kABytes, &tmW, &full[s], kb * 128, row);
      };
      // the first stages' weights, before the wait where that is allowed
      uint32_t pre = 0;
      if (weights_early) {
        while (pre < static_cast<uint32_t>(C::kStages) && work.next(sg))
          for (int kb = sg.kb0; kb < sg.kb1 && pre < static_cast<uint32_t>(C::kStages); ++kb, ++pre) weights(pre, kb);
        work = from_start;
        griddep_wait();
      }
      while (ok && work.next(sg)) {
        const int n16 = (__popcll(tokens_of(sg)) + 15) >> 4;
        for (int kb = sg.kb0; kb < sg.kb1; ++kb, ++it) {
          const int s = it % C::kStages;
          if (it >= static_cast<uint32_t>(C::kStages) && !mbar_wait(&empty[s], ((it / C::kStages) & 1u) ^ 1u)) {
            record_status(kDevTimeoutProducer);
            ok = false;
            break;
          }
          if (it >= pre) weights(it, kb);
          if constexpr (!kBf16) {
            const int row = MODE == kFewDown ? sBase[sg.a] : 0;
            for (int c = 0; c < n16; ++c)
              tma_load_2d(sB + s * C::kBBytes + c * 2048, &tmX, &full[s], kb * 128, row + c * 16);
          }
        }
      }
      // every copy issued must land before the CTA may exit
      for (uint32_t i = (it > static_cast<uint32_t>(C::kStages) ? it - C::kStages : 0); i < it; ++i)
        if (!mbar_wait(&full[i % C::kStages], (i / C::kStages) & 1u)) record_status(kDevTimeoutProducer);
    }
  } else if (warp == kMmaWarp) {
    if (lane == 0) {
      // ================= MMA issuer
      const uint64_t a_desc0 = smem_desc_k_sw128(smem_u32(sA)), b_desc0 = smem_desc_k_sw128(smem_u32(sB));
      uint32_t it = 0;
      bool ok = true;
      while (ok && work.next(sg)) {
        const int n = (__popcll(tokens_of(sg)) + 15) & ~15;
        const uint32_t idesc = idesc_e4m3_f32(128, n);
        for (int kb = sg.kb0; kb < sg.kb1; ++kb, ++it) {
          const int s = it % C::kStages, b = it % C::kNumBuf;
          if (!mbar_wait(&full[s], (it / C::kStages) & 1u) ||
              (it >= static_cast<uint32_t>(C::kNumBuf) && !mbar_wait(&tempty[b], ((it / C::kNumBuf) & 1u) ^ 1u))) {
            record_status(kDevTimeoutMma);
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int t = 0; t < C::kTiles; ++t) {
            const uint32_t d = tmem_base + static_cast<uint32_t>(b * C::kBufCols + t * NT);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_f8f6f4(d, a_desc0 + ((s * C::kABytes + t * 16384 + kk * 32) >> 4),
                         b_desc0 + ((s * C::kBBytes + kk * 32) >> 4), idesc, kk > 0 ? 1u : 0u);
          }
          mma_commit(&empty[s]);
          mma_commit(&tfull[b]);
        }
      }
      mma_commit(mma_done);
      if (!mbar_wait(mma_done, 0)) record_status(kDevTimeoutMma);
    }
  } else if (warp >= kTokWarp0) {
    // ================= token operand and scales of every fourth K block
    uint32_t it = 0;                                                 // blocks before the segment
    uint32_t mine = static_cast<uint32_t>(warp - kTokWarp0);         // this warp's next block
    bool ok = warp - kTokWarp0 < C::kTokWarps;
    while (ok && work.next(sg)) {
      const uint32_t it_end = it + static_cast<uint32_t>(sg.kb1 - sg.kb0);
      const uint64_t m = tokens_of(sg);
      const int n = __popcll(m);
      const uint64_t wrow = (static_cast<uint64_t>(sg.e) * p.NB + (MODE == kFewGateUp ? 2 * sg.j : sg.j)) * p.KB;
      uint32_t sw[C::kTiles];
      auto load_sw = [&](int kb) {
#pragma unroll
        for (int t = 0; t < C::kTiles; ++t)
          sw[t] = load_scale_word(p.Ws, wrow + static_cast<uint64_t>(t) * p.KB + kb, p.fmt);
      };
      // this unit's stage is free
      auto stage_free = [&](uint32_t u) {
        const bool free = u < static_cast<uint32_t>(C::kStages) ||
                          mbar_wait(&empty[u % C::kStages], ((u / C::kStages) & 1u) ^ 1u);
        if (__all_sync(0xFFFFFFFFu, free)) return true;
        if (lane == 0) record_status(kDevTimeoutProducer);
        return false;
      };

      if constexpr (kBf16) {
        // lane: team lane / 8 of a group of four tokens, 16 elements of the
        // 128; 16 tokens (four groups) are in registers at a time
        const int team = lane >> 3, l8 = lane & 7;
        constexpr int kTok = (NT + 31) / 32;
        int tok[kTok];
#pragma unroll
        for (int q = 0; q < kTok; ++q) tok[q] = q * 32 + lane < n ? (kMoe ? nth_bit(m, q * 32 + lane) : q * 32 + lane) : 0;
        uint4 v[4][2];
        auto load16 = [&](int c, int kb) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if (c * 16 + q * 4 >= n) break;
            const int i = c * 16 + q * 4 + team;
            const int t = __shfl_sync(0xFFFFFFFFu, tok[kTok == 1 ? 0 : c >> 1], i & 31);
            v[q][0] = v[q][1] = make_uint4(0, 0, 0, 0);
            if (i < n) {
              const uint4* g = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p.src) +
                                                              static_cast<uint64_t>(t) * p.ld_src + kb * 128 + l8 * 16);
              v[q][0] = __ldg(g);
              v[q][1] = __ldg(g + 1);
            }
          }
        };
        auto store16 = [&](int c, int s) {
          uint8_t* tile = sB + s * C::kBBytes;
          float* sc = sSc + s * C::kTiles * NT;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if (c * 16 + q * 4 >= n) break;
            const int i = c * 16 + q * 4 + team;
            const uint4 x = v[q][0], y = v[q][1];
            uint32_t am = max(absmax_bits8(x), absmax_bits8(y));
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, o));
            uint4 codes;
            float scale;
            auto quant = [&](auto tag) {
              constexpr int F = decltype(tag)::value;
              const GroupScale g = make_scale<F>(am);
              codes.x = quant4<F>(x.x, x.y, g);
              codes.y = quant4<F>(x.z, x.w, g);
              codes.z = quant4<F>(y.x, y.y, g);
              codes.w = quant4<F>(y.z, y.w, g);
              scale = F == 0 ? g.s : scale_value(g.e8, 1);
            };
            if (p.fmt == 0) quant(std::integral_constant<int, 0>{});
            else quant(std::integral_constant<int, 1>{});
            if (i < n) {
              // chunk l8 of row i at l8 ^ (i % 8): the 128-byte swizzle of a TMA tile
              *reinterpret_cast<uint4*>(tile + i * 128 + ((l8 ^ (i & 7)) << 4)) = codes;
              if (l8 == 0) {
#pragma unroll
                for (int t = 0; t < C::kTiles; ++t) sc[t * NT + i] = scale * scale_value(sw[t], p.fmt);
              }
            }
          }
        };
        auto kb_of = [&](uint32_t u) { return sg.kb0 + static_cast<int>(u - it); };
        if (mine < it_end) {
          load16(0, kb_of(mine));
          load_sw(kb_of(mine));
        }
        for (; mine < it_end; mine += C::kTokWarps) {
          const int kb = kb_of(mine);
          const int s = mine % C::kStages;
          if (!stage_free(mine)) {
            ok = false;
            break;
          }
          store16(0, s);
#pragma unroll
          for (int c = 1; c < NT / 16; ++c) {
            if (c * 16 >= n) break;
            load16(c, kb);
            store16(c, s);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&full[s]);
          if (mine + C::kTokWarps < it_end) {
            load16(0, kb + C::kTokWarps);
            load_sw(kb + C::kTokWarps);
          }
        }
      } else {
        // lane: the scales of tokens lane, lane + 32
        constexpr int kTok = (NT + 31) / 32;
        uint32_t sa[kTok];
        const uint64_t pair0 = MODE == kFewDown ? sBase[sg.a] : 0;
        auto load_sa = [&](int kb) {
#pragma unroll
          for (int q = 0; q < kTok; ++q) {
            const int i = q * 32 + lane;
            sa[q] = 0;
            if (i < n) {
              if (MODE == kFewDown)                                  // written by GateUp: a plain load
                sa[q] = reinterpret_cast<const uint32_t*>(p.src_scale)[(pair0 + i) * p.KB + kb];
              else
                sa[q] = load_scale_word(p.src_scale, i + static_cast<uint64_t>(kb) * p.ld_s, p.fmt);
            }
          }
        };
        auto kb_of = [&](uint32_t u) { return sg.kb0 + static_cast<int>(u - it); };
        if (mine < it_end) {
          load_sa(kb_of(mine));
          load_sw(kb_of(mine));
        }
        for (; mine < it_end; mine += C::kTokWarps) {
          const int kb = kb_of(mine);
          const int s = mine % C::kStages;
          if (!stage_free(mine)) {
            ok = false;
            break;
          }
          float* sc = sSc + s * C::kTiles * NT;
          const float w = scale_value(sw[0], p.fmt);
#pragma unroll
          for (int q = 0; q < kTok; ++q) {
            const int i = q * 32 + lane;
            if (i < n) sc[i] = w * (MODE == kFewDown ? __uint_as_float(sa[q]) : scale_value(sa[q], p.fmt));
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&full[s]);
          if (mine + C::kTokWarps < it_end) {
            load_sa(kb + C::kTokWarps);
            load_sw(kb + C::kTokWarps);
          }
        }
      }
      it = it_end;
    }
  } else {
    // ================= promotion and epilogue: thread = weight row
    const int grp = C::kGroups == 1 ? 0 : warp >> 2, quad = warp & 3;
    const int row = quad * 32 + lane;                                // 0..127
    const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
    float* red = sRed + grp * (C::kRedBytes / C::kGroups / 4);
    uint32_t it = 0, meets = 0, segs = 0;
    bool ok = true;
    auto expired = [&] {
      if (lane == 0) record_status(kDevTimeoutEpilogue);
      ok = false;
    };
    // first token of this group's chunk q
    auto chunk0 = [&](int q) { return (q * C::kGroups + grp) * 16; };

    // The ranks' partial sums of 16 tokens t0 + i < n (val[tile][i]): on
    // return the rank that owns a token (token % S) holds the sum over the
    // ranks, added in rank order; the others' entries are left as they were.
    auto meet = [&](float (&val)[C::kTiles][16], int t0, int n) {
#pragma unroll
      for (int c = 0; c < 16 / C::kRedTok; ++c) {
        if (t0 + c * C::kRedTok >= n || !ok) break;
        if (meets > 0 && !__all_sync(0xFFFFFFFFu, mbar_wait_cluster(&red_empty[grp], (meets - 1) & 1u))) {
          expired();
          break;
        }
        // token c * kRedTok + q goes to rank q % S (S divides kRedTok), slot q / S
        const int slots = C::kRedTok >> lgS;
#pragma unroll
        for (int q = 0; q < C::kRedTok; ++q) {
          if (t0 + c * C::kRedTok + q < n) {
            const uint32_t at = static_cast<uint32_t>(((rank * slots + (q >> lgS)) * C::kTiles * 128 + row) * 4);
            const uint32_t to = map_to_rank(smem_u32(red) + at, q & (S - 1));
#pragma unroll
            for (int t = 0; t < C::kTiles; ++t) st_cluster_f32(to + t * 512, val[t][c * C::kRedTok + q]);
          }
        }
        __syncwarp();
        if (lane < S) mbar_arrive_cluster(map_to_rank(smem_u32(&red_full[grp]), lane));
        if (!__all_sync(0xFFFFFFFFu, mbar_wait_cluster(&red_full[grp], meets & 1u))) {
          expired();
          break;
        }
#pragma unroll
        for (int q = 0; q < C::kRedTok; ++q) {
          if ((q & (S - 1)) == rank && t0 + c * C::kRedTok + q < n) {
#pragma unroll
            for (int t = 0; t < C::kTiles; ++t) {
              float sum = 0.0f;
              for (int r = 0; r < S; ++r) sum += red[((r * slots + (q >> lgS)) * C::kTiles + t) * 128 + row];
              val[t][c * C::kRedTok + q] = sum;
            }
          }
        }
        __syncwarp();
        if (lane < S) mbar_arrive_cluster(map_to_rank(smem_u32(&red_empty[grp]), lane));
        ++meets;
      }
    };

    float acc[C::kChunks][C::kTiles][16];
    while (ok && work.next(sg)) {
      const uint64_t m = tokens_of(sg);
      const int n = __popcll(m);
#pragma unroll
      for (int q = 0; q < C::kChunks; ++q)
#pragma unroll
        for (int t = 0; t < C::kTiles; ++t)
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[q][t][i] = 0.0f;
      for (int kb = sg.kb0; kb < sg.kb1; ++kb, ++it) {
        const int b = it % C::kNumBuf, s = it % C::kStages;
        // the scales come from other threads: the stage's full barrier orders them
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(&full[s], (it / C::kStages) & 1u) &&
                                         mbar_wait(&tfull[b], (it / C::kNumBuf) & 1u))) {
          expired();
          break;
        }
        tc_fence_after();
        const float4* sc = reinterpret_cast<const float4*>(sSc + s * C::kTiles * NT);
        // one wait for as many TMEM loads as registers allow
        constexpr int kBatch = C::kTiles == 1 ? C::kChunks : 1;
#pragma unroll
        for (int q0 = 0; q0 < C::kChunks; q0 += kBatch) {
          if (chunk0(q0) >= n) break;
          uint32_t d[kBatch][C::kTiles][16];
#pragma unroll
          for (int q = 0; q < kBatch; ++q) {
            if (chunk0(q0 + q) >= n) break;
#pragma unroll
            for (int t = 0; t < C::kTiles; ++t)
              tmem_ld_32x32b_x16(lane_base + static_cast<uint32_t>(b * C::kBufCols + t * NT + chunk0(q0 + q)), d[q][t]);
          }
          tmem_wait_ld();
#pragma unroll
          for (int q = 0; q < kBatch; ++q) {
            if (chunk0(q0 + q) >= n) break;
#pragma unroll
            for (int t = 0; t < C::kTiles; ++t)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float4 f = sc[(t * NT + chunk0(q0 + q)) / 4 + i];
                float* a = &acc[q0 + q][t][4 * i];
                const uint32_t* x = &d[q][t][4 * i];
                a[0] = __fmaf_rn(__uint_as_float(x[0]), f.x, a[0]);
                a[1] = __fmaf_rn(__uint_as_float(x[1]), f.y, a[1]);
                a[2] = __fmaf_rn(__uint_as_float(x[2]), f.z, a[2]);
                a[3] = __fmaf_rn(__uint_as_float(x[3]), f.w, a[3]);
              }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&tempty[b]);
          mbar_arrive(&empty[s]);
        }
      }
      if (!ok) break;

      if constexpr (MODE != kFewDown) {
        if (S > 1) {
#pragma unroll
          for (int q = 0; q < C::kChunks; ++q)
            if (chunk0(q) < n && ok) meet(acc[q], chunk0(q), n);
          if (!ok) break;
        }
      }
      if constexpr (MODE == kFewGateUp) {
        // h = silu(g) u in fp32, its 1x128 group (the 128 threads' rows)
        // quantized straight from fp32: no rounding to bf16 on the way
        float* am = sAmax + (segs & 1u) * 4 * NT;
#pragma unroll
        for (int q = 0; q < C::kChunks; ++q) {
          if (chunk0(q) >= n) break;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int ti = chunk0(q) + i;
            if (ti < n && (i & (S - 1)) == rank) {
              const float g = acc[q][0][i];
              const float h = __fdiv_rn(g, 1.0f + expf(-g)) * acc[q][1][i];
              acc[q][0][i] = h;
              const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(h) & 0x7FFFFFFFu);
              if (lane == 0) am[quad * NT + ti] = __uint_as_float(top);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&amax_bar[grp]);
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(&amax_bar[grp], segs & 1u))) {
          expired();
          break;
        }
        const uint64_t pair0 = sBase[sg.a];
#pragma unroll
        for (int q = 0; q < C::kChunks; ++q) {
          if (chunk0(q) >= n) break;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int ti = chunk0(q) + i;
            if (ti < n && (i & (S - 1)) == rank) {
              // magnitude bits compare like the values, and a NaN above all of them
              const uint32_t a01 = max(__float_as_uint(am[ti]), __float_as_uint(am[NT + ti]));
              const uint32_t a23 = max(__float_as_uint(am[2 * NT + ti]), __float_as_uint(am[3 * NT + ti]));
              const float scale = scale_of_f32(__uint_as_float(max(a01, a23)), p.fmt);
              const uint64_t r = pair0 + ti;
              FGFP8_DCHECK(r < static_cast<uint64_t>(p.T) * p.topk && sg.j * 128 + row < p.I);
              p.Hq[r * p.I + sg.j * 128 + row] =
                  __nv_cvt_float_to_fp8(__fdiv_rn(acc[q][0][i], scale), __NV_SATFINITE, __NV_E4M3);
              if (row == 0) p.Hs[r * (p.I / 128) + sg.j] = scale;
            }
          }
        }
      } else if constexpr (MODE == kFewDown) {
        // the expert's tokens, weighted, into the block's fp32 sums; a token
        // that names the expert in several slots adds their weights.  The
        // groups hold different tokens of one expert, but a token may change
        // groups from one expert to the next: each expert waits for the last.
        if (C::kGroups > 1 && segs > 0 && !__all_sync(0xFFFFFFFFu, mbar_wait(seg_bar, (segs - 1) & 1u))) {
          expired();
          break;
        }
#pragma unroll
        for (int q = 0; q < C::kChunks; ++q) {
          if (chunk0(q) >= n) break;
          int tok = 0;
          float wt = 0.0f;
          if (lane < 16 && chunk0(q) + lane < n) {
            tok = nth_bit(m, chunk0(q) + lane);
            for (int k = 0; k < p.topk; ++k)
              if (sIds[tok * p.topk + k] == sg.e) wt += sWt[tok * p.topk + k];
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int t = __shfl_sync(0xFFFFFFFFu, tok, i);
            const float w = __shfl_sync(0xFFFFFFFFu, wt, i);
            if (chunk0(q) + i < n) sAcc[t * 128 + row] = __fmaf_rn(w, acc[q][0][i], sAcc[t * 128 + row]);
          }
        }
        if (C::kGroups > 1) {
          __syncwarp();
          if (lane == 0) mbar_arrive(seg_bar);
        }
      } else {
        const int col = sg.j * 128 + row;
        const float bias = load_bias(p.epi, col);
#pragma unroll
        for (int q = 0; q < C::kChunks; ++q) {
          if (chunk0(q) >= n) break;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int t = chunk0(q) + i;
            if (t < n && (i & (S - 1)) == rank) {
              float y = apply_act(acc[q][0][i] + bias, p.epi.act);
              if (p.epi.residual) y += __bfloat162float(p.epi.residual[static_cast<uint64_t>(t) * p.epi.ld_r + col]);
              FGFP8_DCHECK(t < p.T && col < p.N);
              p.Y[static_cast<uint64_t>(t) * p.N + col] = __float2bfloat16_rn(y);
            }
          }
        }
      }
      ++segs;
    }

    if constexpr (MODE == kFewDown) {
      // the block's sums over all experts, residual added, one rounding
      if (C::kGroups > 1 && ok && segs > 0 && !__all_sync(0xFFFFFFFFu, mbar_wait(seg_bar, (segs - 1) & 1u))) expired();
      const int col = cluster * 128 + row;
#pragma unroll
      for (int q = 0; q < C::kChunks; ++q) {
        if (chunk0(q) >= p.T || !ok) break;
        float val[1][16];
#pragma unroll
        for (int i = 0; i < 16; ++i) val[0][i] = sAcc[(chunk0(q) + i) * 128 + row];
        if (S > 1) meet(val, chunk0(q), p.T);
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int t = chunk0(q) + i;
          if (t < p.T && (i & (S - 1)) == rank) {
            float y = val[0][i];
            if (p.epi.residual) y += __bfloat162float(p.epi.residual[static_cast<uint64_t>(t) * p.epi.ld_r + col]);
            FGFP8_DCHECK(col < p.N);
            p.Y[static_cast<uint64_t>(t) * p.N + col] = __float2bfloat16_rn(y);
          }
        }
      }
    }
  }

  // ---- teardown
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (S > 1) cluster_sync();                      // no rank leaves while another may still write to it
  if (warp == kMmaWarp) tmem_dealloc(tmem_base, C::kTmemCols);
}

}  // namespace fgfp8
