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
//   tokens      (4 warps) the token operand of the K blocks in their stages and
//               the products sa * sw.  Up to 16 tokens GateUp (8: Linear)
//               reads bf16 rows, quantizes them and writes the 128-byte-
//               swizzled tile: the rows are L2-resident, and quantizing them
//               again per weight block costs few instructions per 16 KB of
//               weights and saves a kernel.  One warp per block, so that the
//               blocks' loads overlap: the proxy fence before a block is
//               handed over waits for its thread's loads (all four warps on
//               every block: 87 us at 37 x 18432 x 7168, one warp each: 52).
//               With more tokens that arithmetic falls behind the weights
//               (64 tokens x 32 experts: 395 us, from codes 282), so the rows
//               come as codes, by TMA: 16 contiguous rows a copy, or gathered
//               four at a time for an expert's tokens;
//   TMA         (1 warp) the weight tiles;
//   MMA         (1 or 2 warps) owns TMEM, issues the MMAs.
//
// Measured (one B200, back to back in a CUDA graph, weights read once at the
// measured 6.57 TB/s as the floor): 1 token x 8 of 256 experts of 7168 x 2048
// 71 us (floor 53.7), 7 tokens 355 (342), 64 tokens x 32 experts 257 (215);
// linear 1 x 4096 x 4096 7.2 us (2.6), 37 x 18432 x 7168 28 us (20.4).  What
// remains is the start (launch, routing, the first weights' latency: 5 to 8
// us), the gate/up kernel's end (its last epilogues and the hand-over, 5 us),
// and with few blocks the ranks' meeting (2 us).
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
  const void* src_scale;            // codes only: Down fp32 [pair, KB], else MN-major [KB, ld_s] in `fmt`
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
  int withhold = -1;                // self-tests: CTA 0 never requests its withhold-th weight tile
};

template <int MODE, int NT>
struct FewCfg {
  static constexpr int kTiles = MODE == kFewGateUp ? 2 : 1;          // 128-row weight tiles per stage
  static constexpr uint32_t kABytes = kTiles * 128 * 128;
  static constexpr uint32_t kBBytes = NT * 128;
  // The products sa * sw have a ring of their own, so that a stage is free as
  // soon as its MMAs are done.  When a token warp may write block u's, the
  // MMAs of block u - kStages are done, so the promotion has left the pair two
  // before that block's, and with it every block up to u - kStages - 4.
  static constexpr int kScSlots = MODE == kFewGateUp && NT == 16 ? 8 : 16;
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
  static constexpr bool kMoe = MODE != kFewLinear;
  static constexpr uint32_t kMaskBytes = kMoe ? kFewMaxExperts * sizeof(Mask) : 0;
  static constexpr uint32_t kBaseBytes = kMoe ? kFewMaxExperts * 2 : 0;             // first pair of each expert, u16
  static constexpr uint32_t kActBytes = kMoe ? kActive * 2 : 0;                     // active experts, u16
  static constexpr uint32_t kTokBytes = kMoe ? kPairs : 0;                          // token of each pair, u8
  static constexpr uint32_t kWeightBytes = MODE == kFewDown ? kPairs * 4 : 0;       // weight of each pair
  static constexpr uint32_t kAmaxBytes = MODE == kFewGateUp ? kGroups * 2 * 4 * kRedTok * 4 : 0;
  static constexpr uint32_t kBarrierBytes = 384;
  // Two CTAs per SM while the token tile is small: one CTA's ramp and
  // epilogue run under the other's stream.
  static constexpr int kCtas = NT == 16 ? 2 : 1;
  static constexpr uint32_t kBudget = (kCtas == 2 ? 115712u : 232448u) - 1024u;     // after the 1 KB alignment
  static constexpr uint32_t kFixed =
      kScSlots * kScBytes + kRedBytes + kAccBytes + kMaskBytes + kBaseBytes + kActBytes + kTokBytes + kWeightBytes +
      kAmaxBytes + kBarrierBytes;
  static constexpr uint32_t kStageBytes = kABytes + kBBytes;
  static constexpr int kStagesFit = static_cast<int>((kBudget - kFixed) / kStageBytes);
  static constexpr int kStages = kStagesFit > 8 ? 8 : kStagesFit;
  static constexpr size_t kSmemBytes = 1024 + kFixed + static_cast<size_t>(kStages) * kStageBytes;
  // Warps that prepare token operands: stage s belongs to warp s % kTokWarps,
  // so that a warp meets every phase of its stages' barriers in turn.
  static constexpr int kTokWarps = 4;
  // TMEM holds two pairs of K blocks: the promotion takes a pair at a time
  // (one wait for the MMAs and one for the TMEM loads of both; with single
  // blocks its chain of waits took 500 cycles a block, where 16 KB of weights
  // take 540 to 700).
  static constexpr int kNumBuf = 2;
  static constexpr uint32_t kBlockCols = kTiles * NT;
  static constexpr uint32_t kBufCols = 2 * kBlockCols;
  static constexpr uint32_t kTmemCols = kNumBuf * kBufCols;                          // 64 to 512
  // Issuing a block's MMAs, commits and waits takes one warp about 480
  // cycles.  Alone on its SM a CTA wants a block every 540 to 700, so two
  // warps take the pairs in turn (64 tokens x 32 experts: 298 us with one,
  // 283 with two).
  static constexpr int kMmaWarps = NT == 64 ? 2 : 1;
  static constexpr int kThreads = (kEpiWarps + 5 + kMmaWarps) * 32;
  static_assert(kStages >= 3, "pipeline depth");
  static_assert(kScSlots >= kStages + 4, "ring of the scales");
  static_assert(kMmaWarps == 1 || kStages >= 4, "parity waits of the MMA warps");
  static_assert(kTmemCols >= 32 && (kTmemCols & (kTmemCols - 1)) == 0 && kTmemCols * kCtas <= 512, "TMEM columns");
  static_assert((2 * kStages + kScSlots + 2 * kNumBuf + 9) * 8 + 16 <= kBarrierBytes, "barrier area");
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
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

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

// Scale s of a group whose amax is a full fp32 number, and r = RN(1/s):
// max(amax, 1e-4) / 448, or the smallest power of two not below that.  The
// quotients are Markstein's FMA form, as in make_scale and quant4; the
// division routine's slow path (values of slots without a token, say) took
// most of the epilogue's time.
__device__ __forceinline__ float scale_of_f32(float amax, int fmt, float& r) {
  const float a = amax < 1e-4f ? 1e-4f : amax;
  constexpr float kR448 = 1.0f / 448.0f;
  const float q0 = __fmul_rn(a, kR448);
  float s = __fmaf_rn(__fmaf_rn(-q0, 448.0f, a), kR448, q0);
  if (fmt != 0) {
    uint32_t b = __float_as_uint(s), e = b >> 23;
    if ((b & 0x7FFFFFu) != 0u && e < 255u) e += 1u;
    s = scale_value(e, 1);
  }
  r = __frcp_rn(s);
  return s;
}
__device__ __forceinline__ uint8_t quant_f32(float x, float s, float r) {
  const float q0 = __fmul_rn(x, r);
  return __nv_cvt_float_to_fp8(__fmaf_rn(__fmaf_rn(-q0, s, x), r, q0), __NV_SATFINITE, __NV_E4M3);
}

// ------------------------------------------------------------ work of a CTA
// A segment: K blocks [kb0, kb1) of one expert's weight rows.
struct FewSeg {
  int a, e;                         // position in the active list, expert
  int j;                            // GateUp: 128-wide block of I; else the 128-row block of N
  int kb0, kb1;
  bool joint;                       // the cluster's ranks share the piece, each a part of its K
};

// The segments of one CTA, the same sequence for every role.
//   GateUp  items (a, j), each CTA one of its own per round.  What is left for
//           the last round, if it is at most one item per cluster, the ranks
//           share: r takes the r-th of S parts of K (512 items on 148 CTAs: the
//           last round of 68 took as long as a full one)
//   Down    the cluster's block of 128 output columns: the (a, kb) blocks of
//           all active experts in one line, cut into S equal ranges
//   Linear  the cluster's block of 128 output columns, rank r its S-th of K
template <int MODE>
struct FewIter {
  int pos, end, KB, NJ, j, rank, lgS, cluster, ctas;
  const uint16_t* act;
  __device__ FewIter(const FewArgs& p, int active, const uint16_t* act_, int rank_, int cluster_) {
    act = act_;
    KB = p.KB;
    NJ = p.I / 128;
    j = cluster = cluster_;
    rank = rank_;
    lgS = p.lgS;
    ctas = gridDim.x;
    pos = 0, end = 1;
    if (MODE == kFewGateUp) {
      end = active * NJ;                              // items; pos: the round's first
    } else if (MODE == kFewDown) {
      const int units = active * KB;                  // at most 2^9 experts x 2^13 blocks
      pos = units * rank >> lgS;
      end = units * (rank + 1) >> lgS;
    }
  }
  __device__ bool next(FewSeg& s) {
    if (pos >= end) return false;
    s.joint = true;
    if (MODE == kFewGateUp) {
      const int left = end - pos;
      s.joint = left <= ctas >> lgS && lgS > 0;
      const int mine = s.joint ? cluster : (cluster << lgS) + rank;
      if (mine >= left) return false;
      s.a = (pos + mine) / NJ;
      s.j = pos + mine - s.a * NJ;
      s.e = act[s.a];
      s.kb0 = s.joint ? KB * rank >> lgS : 0;
      s.kb1 = s.joint ? KB * (rank + 1) >> lgS : KB;
      pos += s.joint ? left : ctas;
    } else if (MODE == kFewDown) {
      s.a = pos / KB;
      s.e = act[s.a];
      s.j = j;
      s.kb0 = pos - s.a * KB;
      s.kb1 = s.kb0 + (end - pos) < KB ? s.kb0 + (end - pos) : KB;
      pos += s.kb1 - s.kb0;
    } else {
      s.a = 0, s.e = 0, s.j = j;
      s.kb0 = KB * rank >> lgS, s.kb1 = KB * (rank + 1) >> lgS;
      pos = end;
    }
    return true;
  }
};

// A mask of one bit per token: those below t.
template <typename M>
__device__ __forceinline__ M bits_below(int t) {
  return (M(1) << t) - M(1);
}

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(p));
  return p != 0;
}

template <int MODE, int NT, bool kBf16>
__global__ void __launch_bounds__(FewCfg<MODE, NT>::kThreads, FewCfg<MODE, NT>::kCtas)
    few_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
               const __grid_constant__ FewArgs p) {
  using C = FewCfg<MODE, NT>;
  using Mask = typename C::Mask;
  constexpr bool kMoe = C::kMoe;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = sA + C::kStages * C::kABytes;
  float* sSc = reinterpret_cast<float*>(sB + C::kStages * C::kBBytes);             // [slot][tile][NT]
  float* sAcc = sSc + C::kScSlots * C::kTiles * NT;                                // Down: [token][128]
  float* sRed = sAcc + C::kAccBytes / 4;                                           // [group][rank][slot][tile][128]
  Mask* sMask = reinterpret_cast<Mask*>(sRed + C::kRedBytes / 4);                  // tokens of each expert
  float* sWt = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(sMask) + C::kMaskBytes);
  float* sAmax = sWt + C::kWeightBytes / 4;                                        // GateUp: [group][2][4][kRedTok]
  uint64_t* full = reinterpret_cast<uint64_t*>(sAmax + C::kAmaxBytes / 4);
  uint64_t* empty = full + C::kStages;
  uint64_t* tfull = empty + C::kStages;
  uint64_t* tempty = tfull + C::kNumBuf;
  uint64_t* mma_done = tempty + C::kNumBuf;
  uint64_t* red_full = mma_done + 2;
  uint64_t* red_empty = red_full + 2;
  uint64_t* amax_bar = red_empty + 2;
  uint64_t* seg_bar = amax_bar + 2;
  uint64_t* sc_full = seg_bar + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sc_full + C::kScSlots);
  uint16_t* sBase = reinterpret_cast<uint16_t*>(reinterpret_cast<uint8_t*>(full) + C::kBarrierBytes);
  uint16_t* sAct = sBase + C::kBaseBytes / 2;
  uint8_t* sTok = reinterpret_cast<uint8_t*>(sAct + C::kActBytes / 2);
  __shared__ int s_count[2][kFewMaxExperts / 32];                                  // per 32 experts: active, pairs
  __shared__ int s_active;                                                         // experts with tokens

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kTokWarp0 = C::kEpiWarps, kTmaWarp = kTokWarp0 + 4, kMmaWarp = kTmaWarp + 1;
  const int lgS = p.lgS, S = 1 << lgS;
  const int rank = S > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int cluster = static_cast<int>(blockIdx.x) >> lgS;

  if (tid == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1 + 1);                 // the TMA warp and the block's token warp
      mbar_init(&empty[s], 1);                    // the MMAs
    }
    for (int s = 0; s < C::kScSlots; ++s) mbar_init(&sc_full[s], 1);
    for (int b = 0; b < C::kNumBuf; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], C::kEpiWarps);
    }
    for (int w = 0; w < 2; ++w) mbar_init(&mma_done[w], 1);
    for (int g = 0; g < 2; ++g) {
      const int warps = MODE == kFewDown ? C::kEpiWarps : 4;         // Down: the groups meet together
      mbar_init(&red_full[g], warps * S);
      mbar_init(&red_empty[g], warps * S);
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

  // GateUp from bf16 rows reads the routing that the preceding grid may have
  // written, and lets Down start as soon as every CTA here has passed its
  // wait: Down's CTAs then request weights while the last CTAs here finish.
  // GateUp from codes follows the quantizer, which started after all earlier
  // work: the routing and the weights are there, only the codes are not.  So
  // for Down the routing is complete before it starts, and only H and the
  // output wait for GateUp.
  if (MODE == kFewGateUp && kBf16) griddep_wait();
  griddep_launch_dependents();                    // the others' dependents wait before they touch memory
  if constexpr (kMoe) {
    // sMask[e]: the tokens routed to e; sAct: the experts with any, ascending;
    // pair sBase[e] + i: e's i-th token, its weight the sum over the token's
    // slots that name e
    const int P = p.T * p.topk;
    if constexpr (MODE == kFewDown)
      for (int i = tid; i < NT * 128; i += C::kThreads) sAcc[i] = 0.0f;
    if (NT == 16 && P <= 32) {
      // one warp, a lane per slot, no shared-memory passes (the general form's
      // five took 2 us of a single token's 75)
      if (warp == kTmaWarp) {
        const int id = lane < P ? __ldg(p.ids + lane) : -1;
        const float w = MODE == kFewDown && lane < P ? __ldg(p.wts + lane) : 0.0f;
        const int t = lane / p.topk;
        const bool in = id >= 0 && id < p.E;
        if (id >= p.E && blockIdx.x == 0) record_status(kDevBadExpert);
        const uint32_t below = (1u << lane) - 1u;
        const uint32_t ins = __ballot_sync(0xFFFFFFFFu, in);
        const uint32_t same_e = __match_any_sync(0xFFFFFFFFu, id) & ins;              // slots of this expert
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, id * 32 + t) & same_e;    // and of this token (t < 32)
        const bool first = in && (same & below) == 0u;
        const uint32_t firsts = __ballot_sync(0xFFFFFFFFu, first);
        const bool leads = in && (same_e & below) == 0u;
        const uint32_t leaders = __ballot_sync(0xFFFFFFFFu, leads);
        const int count = __popc(same_e & firsts);
        int a = 0, base = 0;                     // experts and pairs before this one
        float sum = 0.0f;
        uint32_t tokens = 0u;
        for (int o = 0; o < P; ++o) {
          const int id_o = __shfl_sync(0xFFFFFFFFu, id, o), n_o = __shfl_sync(0xFFFFFFFFu, count, o);
          const int t_o = __shfl_sync(0xFFFFFFFFu, t, o);
          const float w_o = __shfl_sync(0xFFFFFFFFu, w, o);
          const bool less = ((leaders >> o) & 1u) && id_o < id;
          a += less ? 1 : 0;
          base += less ? n_o : 0;
          tokens |= ((same_e >> o) & 1u) << t_o;
          if ((same >> o) & 1u) sum += w_o;
        }
        if (leads) {
          sAct[a] = static_cast<uint16_t>(id);
          sBase[id] = static_cast<uint16_t>(base);
          sMask[id] = tokens;
        }
        if (first) {
          const int at = base + __popc(same_e & firsts & below);
          sTok[at] = static_cast<uint8_t>(t);
          if constexpr (MODE == kFewDown) sWt[at] = sum;
        }
        if (lane == 0) s_active = __popc(leaders);
      }
    } else {
      for (int e = tid; e < p.E; e += C::kThreads) sMask[e] = 0;
      __syncthreads();
      for (int i = tid; i < P; i += C::kThreads) {
        const int id = __ldg(p.ids + i);
        if (id >= 0 && id < p.E) atomicOr(sMask + id, Mask(1) << (i / p.topk));
        if (id >= p.E && blockIdx.x == 0) record_status(kDevBadExpert);
      }
      __syncthreads();
      const int chunks = (p.E + 31) >> 5;
      auto mask_of = [&](int e) { return e < p.E ? sMask[e] : Mask(0); };
      for (int c = warp; c < chunks; c += C::kThreads / 32) {
        const int k = __popcll(mask_of(c * 32 + lane));
        const uint32_t on = __ballot_sync(0xFFFFFFFFu, k != 0);
        const int pairs = __reduce_add_sync(0xFFFFFFFFu, k);
        if (lane == 0) s_count[0][c] = __popc(on), s_count[1][c] = pairs;
      }
      __syncthreads();
      for (int c = warp; c < chunks; c += C::kThreads / 32) {
        const int k = __popcll(mask_of(c * 32 + lane));
        const uint32_t on = __ballot_sync(0xFFFFFFFFu, k != 0);
        int incl = k;
  #pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
          if (lane >= d) incl += o;
        }
        // chunks before this one (at most 16)
        const int na = __reduce_add_sync(0xFFFFFFFFu, lane < c ? s_count[0][lane & 15] : 0);
        const int np = __reduce_add_sync(0xFFFFFFFFu, lane < c ? s_count[1][lane & 15] : 0);
        if (k != 0) {
          sAct[na + __popc(on & ((1u << lane) - 1u))] = static_cast<uint16_t>(c * 32 + lane);
          sBase[c * 32 + lane] = static_cast<uint16_t>(np + incl - k);
        }
      }
      __syncthreads();
      if (tid == 0) {
        int all = 0;
        for (int c = 0; c < chunks; ++c) all += s_count[0][c];
        s_active = all;
      }
      for (int i = tid; i < P; i += C::kThreads) {
        const int id = __ldg(p.ids + i);
        if (id < 0 || id >= p.E) continue;
        const int t = i / p.topk, j = i - t * p.topk;
        bool first = true;
        for (int k = 0; k < j; ++k) first = first && __ldg(p.ids + t * p.topk + k) != id;
        if (!first) continue;
        const int at = sBase[id] + __popcll(sMask[id] & bits_below<Mask>(t));
        FGFP8_DCHECK(at < C::kPairs);
        sTok[at] = static_cast<uint8_t>(t);
        if constexpr (MODE == kFewDown) {
          float w = __ldg(p.wts + i);
          for (int k = j + 1; k < p.topk; ++k)
            if (__ldg(p.ids + t * p.topk + k) == id) w += __ldg(p.wts + t * p.topk + k);
          sWt[at] = w;
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (S > 1) cluster_arrive();                    // this CTA's barriers exist; the promotion warps wait for the others'
  const uint32_t tmem_base = *tmem_slot;
  FewIter<MODE> work(p, kMoe ? s_active : 1, sAct, rank, cluster);
  FewSeg sg{};
  auto count_of = [&](const FewSeg& s) -> int {   // tokens of a segment
    if constexpr (kMoe) return __popcll(sMask[s.e]);
    return p.T;
  };
  auto pair0_of = [&](const FewSeg& s) -> int {   // their first pair, or row
    if constexpr (kMoe) return sBase[s.e];
    return 0;
  };
  const bool weights_early = MODE == kFewDown || (MODE == kFewGateUp && !kBf16) || (MODE == kFewLinear && p.early);
  if (!(warp == kTmaWarp && weights_early)) griddep_wait();

  if (warp == kTmaWarp) {
    if (lane == 0) {
      // ================= weight tiles
      uint32_t it = 0;
      bool ok = true;
      while (ok && work.next(sg)) {
        const int row = (sg.e * p.NB + (MODE == kFewGateUp ? 2 * sg.j : sg.j)) * 128;
        for (int kb = sg.kb0; kb < sg.kb1; ++kb, ++it) {
          const int s = it % C::kStages;
          if (it >= static_cast<uint32_t>(C::kStages) && !mbar_wait(&empty[s], ((it / C::kStages) & 1u) ^ 1u)) {
            record_status(kDevTimeoutProducer);
            ok = false;
            break;
          }
          if (blockIdx.x == 0 && static_cast<int>(it) == p.withhold) continue;
          mbar_arrive_expect_tx(&full[s], C::kABytes);
          tma_load_2d(sA + s * C::kABytes, &tmW, &full[s], kb * 128, row);
        }
      }
      // every copy issued must land before the CTA may exit
      for (uint32_t i = (it > static_cast<uint32_t>(C::kStages) ? it - C::kStages : 0); i < it; ++i)
        if (!mbar_wait(&full[i % C::kStages], (i / C::kStages) & 1u)) record_status(kDevTimeoutProducer);
    }
  } else if (warp >= kMmaWarp) {
    // ================= MMA issuers, a pair of K blocks each in turn: the whole
    // warp keeps the loop's state uniform, one elected lane issues.  The wait
    // for the pair's TMEM buffer also tells that every block before the other
    // warp's current pair has been full, so that the parity of `full` is not
    // mistaken for the one before the last.
    const uint32_t me = static_cast<uint32_t>(warp - kMmaWarp);
    const uint64_t a_desc0 = smem_desc_k_sw128(smem_u32(sA)), b_desc0 = smem_desc_k_sw128(smem_u32(sB));
    uint32_t it = 0, pairs = 0;
    bool ok = true;
    while (ok && work.next(sg)) {
      const int n = __shfl_sync(0xFFFFFFFFu, (count_of(sg) + 15) & ~15, 0);
      const uint32_t idesc = idesc_e4m3_f32(128, n);
      for (int kb = sg.kb0; kb < sg.kb1 && ok; kb += 2, ++pairs) {
        const int b = pairs % C::kNumBuf;
        const int blocks = sg.kb1 - kb < 2 ? 1 : 2;
        if (C::kMmaWarps > 1 && (pairs & 1u) != me) {
          it += blocks;
          continue;
        }
        bool got = pairs < static_cast<uint32_t>(C::kNumBuf) || mbar_wait(&tempty[b], ((pairs / C::kNumBuf) & 1u) ^ 1u);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h == blocks) break;
          const int s = it % C::kStages;
          got = got && mbar_wait(&full[s], (it / C::kStages) & 1u);
          if (!__all_sync(0xFFFFFFFFu, got)) {
            if (lane == 0) record_status(kDevTimeoutMma);
            ok = false;
            break;
          }
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int t = 0; t < C::kTiles; ++t) {
              const uint32_t d = tmem_base + static_cast<uint32_t>(b * C::kBufCols + h * C::kBlockCols + t * NT);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_f8f6f4(d, a_desc0 + ((s * C::kABytes + t * 16384 + kk * 32) >> 4),
                           b_desc0 + ((s * C::kBBytes + kk * 32) >> 4), idesc, kk > 0 ? 1u : 0u);
            }
            mma_commit(&empty[s]);
            if (h + 1 == blocks) mma_commit(&tfull[b]);
          }
          __syncwarp();
          ++it;
        }
      }
    }
    if (elect_one()) mma_commit(&mma_done[me]);
    __syncwarp();
    if (!mbar_wait(&mma_done[me], 0) && lane == 0) record_status(kDevTimeoutMma);
  } else if (warp >= kTokWarp0) {
    // ================= token operand and scales of this warp's K blocks
    uint32_t it = 0;                                                 // blocks before the segment
    const uint32_t me = static_cast<uint32_t>(warp - kTokWarp0);
    auto mine_from = [&](uint32_t u) {                               // this warp's first block from u on
      while ((u % C::kStages) % C::kTokWarps != me) ++u;
      return u;
    };
    bool ok = me < static_cast<uint32_t>(C::kStages);                // with few stages a warp may have none
    uint32_t mine = ok ? mine_from(0) : 0;
    while (ok && work.next(sg)) {
      const uint32_t it_end = it + static_cast<uint32_t>(sg.kb1 - sg.kb0);
      const int n = count_of(sg), pair0 = pair0_of(sg);
      const uint64_t wrow = (static_cast<uint64_t>(sg.e) * p.NB + (MODE == kFewGateUp ? 2 * sg.j : sg.j)) * p.KB;
      auto kb_of = [&](uint32_t u) { return sg.kb0 + static_cast<int>(u - it); };
      uint32_t sw[C::kTiles];
      auto load_sw = [&](int kb) {
#pragma unroll
        for (int t = 0; t < C::kTiles; ++t)
          sw[t] = load_scale_word(p.Ws, wrow + static_cast<uint64_t>(t) * p.KB + kb, p.fmt);
      };
      // block u's stage is free
      auto stage_free = [&](uint32_t u) {
        const bool free = u < static_cast<uint32_t>(C::kStages) ||
                          mbar_wait(&empty[u % C::kStages], ((u / C::kStages) & 1u) ^ 1u);
        if (__all_sync(0xFFFFFFFFu, free)) return true;
        if (lane == 0) record_status(kDevTimeoutProducer);
        return false;
      };

      if constexpr (kBf16) {
        // lane: team lane / 8 of four, one token per team and pass, 16 of the
        // token's 128 elements.  Four passes together, so that their loads and
        // reductions overlap, or one for up to four tokens.
        const int team = lane >> 3, l8 = lane & 7;
        static_assert(NT == 16, "wider tiles take codes");
        uint4 v[4][2];
        auto load = [&](auto passes, int kb) {
          constexpr int P = decltype(passes)::value;
#pragma unroll
          for (int q = 0; q < P; ++q) {
            const int i = q * 4 + team;
            v[q][0] = v[q][1] = make_uint4(0, 0, 0, 0);
            if (i < n) {
              const int t = kMoe ? sTok[pair0 + i] : i;
              const uint4* g = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p.src) +
                                                              static_cast<uint64_t>(t) * p.ld_src + kb * 128 + l8 * 16);
              v[q][0] = __ldg(g);
              v[q][1] = __ldg(g + 1);
            }
          }
        };
        auto store = [&](auto passes, auto fmt, int s, float* sc) {
          constexpr int P = decltype(passes)::value, F = decltype(fmt)::value;
          uint8_t* tile = sB + s * C::kBBytes;
          uint32_t am[P];
#pragma unroll
          for (int q = 0; q < P; ++q) am[q] = max(absmax_bits8(v[q][0]), absmax_bits8(v[q][1]));
#pragma unroll
          for (int o = 1; o < 8; o <<= 1)
#pragma unroll
            for (int q = 0; q < P; ++q) am[q] = max(am[q], __shfl_xor_sync(0xFFFFFFFFu, am[q], o));
#pragma unroll
          for (int q = 0; q < P; ++q) {
            const int i = q * 4 + team;
            const GroupScale g = make_scale<F>(am[q]);
            uint4 codes;
            codes.x = quant4<F>(v[q][0].x, v[q][0].y, g);
            codes.y = quant4<F>(v[q][0].z, v[q][0].w, g);
            codes.z = quant4<F>(v[q][1].x, v[q][1].y, g);
            codes.w = quant4<F>(v[q][1].z, v[q][1].w, g);
            const float scale = F == 0 ? g.s : scale_value(g.e8, 1);
            if (i < n) {
              // chunk l8 of row i at l8 ^ (i % 8): the 128-byte swizzle of a TMA tile
              *reinterpret_cast<uint4*>(tile + i * 128 + ((l8 ^ (i & 7)) << 4)) = codes;
              if (l8 == 0) {
#pragma unroll
                for (int t = 0; t < C::kTiles; ++t) sc[t * NT + i] = scale * scale_value(sw[t], F);
              }
            }
          }
        };
        using One = std::integral_constant<int, 1>;
        using Four = std::integral_constant<int, 4>;
        using F32 = std::integral_constant<int, 0>;
        using E8 = std::integral_constant<int, 1>;
        auto load_all = [&](int kb) {
          if (n > 4) load(Four{}, kb);
          else load(One{}, kb);
          load_sw(kb);
        };
        auto store_all = [&](int s, float* sc) {
          if (n > 4) {
            if (p.fmt == 0) store(Four{}, F32{}, s, sc);
            else store(Four{}, E8{}, s, sc);
          } else {
            if (p.fmt == 0) store(One{}, F32{}, s, sc);
            else store(One{}, E8{}, s, sc);
          }
        };
        if (mine < it_end) load_all(kb_of(mine));
        while (mine < it_end) {
          const int kb = kb_of(mine);
          const uint32_t next = mine_from(mine + 1);
          const int s = mine % C::kStages;
          if (!stage_free(mine)) {
            ok = false;
            break;
          }
          float* sc = sSc + (mine % C::kScSlots) * C::kTiles * NT;
          store_all(s, sc);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&full[s]);
            mbar_arrive(&sc_full[mine % C::kScSlots]);
          }
          if (next < it_end) load_all(kb_of(next));
          mine = next;
        }
      } else {
        // lane: the scales of tokens lane, lane + 32.  Lane 0 requests the rows
        // where they are contiguous, 16 at a time; GateUp's are anyone's rows
        // of X, and lane g requests rows 4 g .. 4 g + 3 in one gather (the last
        // token's again past the end).
        constexpr int kTok = (NT + 31) / 32;
        const int n16 = (n + 15) >> 4;
        uint32_t sa[kTok];
        int tok[kTok];
#pragma unroll
        for (int q = 0; q < kTok; ++q)
          tok[q] = MODE == kFewGateUp && q * 32 + lane < n ? sTok[pair0 + q * 32 + lane] : q * 32 + lane;
        int four[4];
        const int n4 = (n + 3) >> 2;
        if constexpr (MODE == kFewGateUp) {
#pragma unroll
          for (int k = 0; k < 4; ++k) four[k] = sTok[pair0 + (4 * lane + k < n ? 4 * lane + k : n - 1)];
        }
        auto load_sa = [&](int kb) {
#pragma unroll
          for (int q = 0; q < kTok; ++q) {
            const int i = q * 32 + lane;
            sa[q] = 0;
            if (i < n) {
              if (MODE == kFewDown)                                  // written by GateUp: a plain load
                sa[q] = reinterpret_cast<const uint32_t*>(p.src_scale)[static_cast<uint64_t>(pair0 + i) * p.KB + kb];
              else
                sa[q] = load_scale_word(p.src_scale, tok[q] + static_cast<uint64_t>(kb) * p.ld_s, p.fmt);
            }
          }
        };
        if (mine < it_end) {
          load_sa(kb_of(mine));
          load_sw(kb_of(mine));
        }
        while (mine < it_end) {
          const int kb = kb_of(mine);
          const uint32_t next = mine_from(mine + 1);
          const int s = mine % C::kStages;
          if (!stage_free(mine)) {
            ok = false;
            break;
          }
          float* sc = sSc + (mine % C::kScSlots) * C::kTiles * NT;
          uint8_t* tile = sB + s * C::kBBytes;
          // the rows first: their latency and the scales' overlap
          if (MODE == kFewGateUp) {
            if (lane == 0) mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(n4 * 512));
            __syncwarp();
            if (lane < n4)
              tma_gather4_2d(tile + lane * 512, &tmX, &full[s], kb * 128, four[0], four[1], four[2], four[3]);
          } else if (lane == 0) {
            mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(n16 * 2048));
            for (int c = 0; c < n16; ++c) tma_load_2d(tile + c * 2048, &tmX, &full[s], kb * 128, pair0 + c * 16);
          }
#pragma unroll
          for (int q = 0; q < kTok; ++q) {
            const int i = q * 32 + lane;
            const float a = MODE == kFewDown ? __uint_as_float(sa[q]) : scale_value(sa[q], p.fmt);
            if (i < n) {
#pragma unroll
              for (int t = 0; t < C::kTiles; ++t) sc[t * NT + i] = a * scale_value(sw[t], p.fmt);
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sc_full[mine % C::kScSlots]);
          if (next < it_end) {
            load_sa(kb_of(next));
            load_sw(kb_of(next));
          }
          mine = next;
        }
      }
      it = it_end;
    }
    if constexpr (!kBf16) {
      // Every copy that this warp issued must land before the CTA may exit.
      // The TMA warp waits for its own blocks only: behind an expired wait,
      // with two MMA warps, this warp may have come further.
      if (lane == 0)
        for (uint32_t u = mine > static_cast<uint32_t>(C::kStages) ? mine - C::kStages : 0; u < mine; ++u)
          if ((u % C::kStages) % C::kTokWarps == me && !mbar_wait(&full[u % C::kStages], (u / C::kStages) & 1u))
            record_status(kDevTimeoutProducer);
    }
  } else {
    // ================= promotion and epilogue: thread = weight row
    const int grp = C::kGroups == 1 ? 0 : warp >> 2, quad = warp & 3;
    const int row = quad * 32 + lane;                                // 0..127
    const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
    float* red = sRed + grp * (C::kRedBytes / C::kGroups / 4);
    constexpr int kSubs = C::kChunks * 16 / C::kRedTok;              // meetings of a full tile
    // How the current piece's tokens are shared: by the cluster's ranks, or (a
    // GateUp item of this CTA alone) not at all.
    int slots = C::kRedTok >> lgS, lgW = lgS, who = rank;            // tokens of a meeting per rank
    uint32_t it = 0, pairs = 0, meets = 0, segs = 0, quants = 0;
    bool ok = true;
    auto expired = [&] {
      if (lane == 0) record_status(kDevTimeoutEpilogue);
      ok = false;
    };
    // first token of this group's chunk q, and of its meeting c
    auto chunk0 = [&](int q) { return (q * C::kGroups + grp) * 16; };
    auto sub0 = [&](int c) { return chunk0(c * C::kRedTok / 16) + c * C::kRedTok % 16; };
    // A rank's token in slot k of a meeting is who + k 2^lgW (2^lgW divides kRedTok).
    auto own_of = [&](int c, int n) {                                // slots with a token below n
      const int left = n - sub0(c) - who;
      const int k = left <= 0 ? 0 : (left + (1 << lgW) - 1) >> lgW;
      return k < slots ? k : slots;
    };

    // One meeting of the ranks: each thread's partial sums x of its row for
    // kRedTok tokens, `count` of them real, go to the tokens' owners, token q
    // to rank q % S, slot q / S; back come the sums over the ranks, added in
    // rank order, of this rank's tokens in their slots.  A meeting is counted
    // before the waits that may expire: the cluster's first phase, which every
    // thread arrives at once, is waited for at the first meeting, or, where
    // none was begun (meets == 0), at the role's end, and never twice.
    auto meet = [&](float (&x)[C::kTiles][C::kRedTok], int count) {
      const uint32_t before = meets++;
      if (before == 0) cluster_wait();                               // the others' barriers exist
      if (before > 0 && !__all_sync(0xFFFFFFFFu, mbar_wait_cluster(&red_empty[grp], (before - 1) & 1u))) {
        expired();
        return;
      }
#pragma unroll
      for (int q = 0; q < C::kRedTok; ++q) {
        if (q >= count) break;
        const int at = ((rank * slots + (q >> lgS)) * C::kTiles) * 128 + row;
        const uint32_t to = map_to_rank(smem_u32(red + at), q & (S - 1));
#pragma unroll
        for (int t = 0; t < C::kTiles; ++t) st_cluster_f32(to + t * 512, x[t][q]);
      }
      __syncwarp();
      if (lane < S) mbar_arrive_cluster(map_to_rank(smem_u32(&red_full[grp]), lane));
      if (!__all_sync(0xFFFFFFFFu, mbar_wait_cluster(&red_full[grp], before & 1u))) {
        expired();
        return;
      }
#pragma unroll
      for (int t = 0; t < C::kTiles; ++t)
#pragma unroll
        for (int k = 0; k < C::kRedTok; ++k) x[t][k] = 0.0f;
#pragma unroll 1
      for (int r = 0; r < S; ++r) {
        const float* from = red + r * slots * C::kTiles * 128 + row;
#pragma unroll
        for (int k = 0; k < C::kRedTok / 2; ++k)                     // S >= 2
          if (k < slots) {
#pragma unroll
            for (int t = 0; t < C::kTiles; ++t) x[t][k] += from[(k * C::kTiles + t) * 128];
          }
      }
      __syncwarp();
      if (lane < S) mbar_arrive_cluster(map_to_rank(smem_u32(&red_empty[grp]), lane));
    };

    // Output rows (Linear, Down): this rank's tokens of meeting c, all in
    // flight together (one token after the other took 500 cycles each).  Their
    // residuals are loaded a meeting ahead, the first one's before the K loop.
    const int col = (MODE == kFewGateUp ? 0 : cluster) * 128 + row;
    float bias = 0.0f;
    uint16_t res[C::kRedTok];                                        // of the meeting to come
    auto load_res = [&](int c) {
      const int own = c < kSubs ? own_of(c, p.T) : 0;
      const uint16_t* from = reinterpret_cast<const uint16_t*>(p.epi.residual) +
                             static_cast<uint64_t>(sub0(c) + rank) * p.epi.ld_r + col;
#pragma unroll
      for (int k = 0; k < C::kRedTok; ++k) res[k] = 0;
      if (p.epi.residual == nullptr) return;
#pragma unroll
      for (int k = 0; k < C::kRedTok; ++k)
        if (k < own) res[k] = from[(static_cast<uint64_t>(k) << lgS) * p.epi.ld_r];
    };
    auto finish_rows = [&](int c, float (&x)[C::kRedTok]) {
      const int own = own_of(c, p.T);
      if constexpr (MODE == kFewLinear) {
#pragma unroll
        for (int k = 0; k < C::kRedTok; ++k) x[k] += bias;
        apply_act_n(x, p.epi.act);
      }
#pragma unroll
      for (int k = 0; k < C::kRedTok; ++k) x[k] += __uint_as_float(static_cast<uint32_t>(res[k]) << 16);
      load_res(c + 1);
      FGFP8_DCHECK(col < p.N && (own == 0 || sub0(c) + rank + ((own - 1) << lgS) < p.T));
      __nv_bfloat16* to = p.Y + static_cast<uint64_t>(sub0(c) + rank) * p.N + col;
#pragma unroll
      for (int k = 0; k < C::kRedTok; ++k)
        if (k < own) to[(static_cast<uint64_t>(k) << lgS) * p.N] = __float2bfloat16_rn(x[k]);
    };
    if constexpr (MODE != kFewGateUp) {
      load_res(0);
      if (MODE == kFewLinear) bias = load_bias(p.epi, col);
    }

    float acc[C::kChunks][C::kTiles][16];
    while (ok && work.next(sg)) {
      const int n = count_of(sg), pair0 = pair0_of(sg);
      if (MODE == kFewGateUp) {
        lgW = sg.joint ? lgS : 0;
        who = sg.joint ? rank : 0;
        slots = C::kRedTok >> lgW;
      }
#pragma unroll
      for (int q = 0; q < C::kChunks; ++q)
#pragma unroll
        for (int t = 0; t < C::kTiles; ++t)
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[q][t][i] = 0.0f;
      for (int kb = sg.kb0; kb < sg.kb1; kb += 2, ++pairs) {
        const int b = pairs % C::kNumBuf;
        const int blocks = sg.kb1 - kb < 2 ? 1 : 2;
        const int s0 = it % C::kScSlots, s1 = (it + 1) % C::kScSlots;
        bool got = mbar_wait(&tfull[b], (pairs / C::kNumBuf) & 1u) && mbar_wait(&sc_full[s0], (it / C::kScSlots) & 1u);
        if (blocks == 2) got = got && mbar_wait(&sc_full[s1], ((it + 1) / C::kScSlots) & 1u);
        if (!__all_sync(0xFFFFFFFFu, got)) {
          expired();
          break;
        }
        tc_fence_after();
        // One wait for both blocks' TMEM loads of a chunk.  Of a single block
        // the second half is another pair's stale partial: not added.
#pragma unroll
        for (int q = 0; q < C::kChunks; ++q) {
          if (chunk0(q) >= n) break;
#pragma unroll
          for (int t = 0; t < C::kTiles; ++t) {
            uint32_t d[2][16];
#pragma unroll
            for (int h = 0; h < 2; ++h)
              tmem_ld_32x32b_x16(lane_base + static_cast<uint32_t>(b * C::kBufCols + h * C::kBlockCols + t * NT + chunk0(q)),
                                 d[h]);
            tmem_wait_ld();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (h == blocks) break;
              const float4* sc = reinterpret_cast<const float4*>(sSc + (h == 0 ? s0 : s1) * C::kTiles * NT + t * NT + chunk0(q));
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float4 f = sc[i];
                float* a = &acc[q][t][4 * i];
                const uint32_t* v = &d[h][4 * i];
                a[0] = __fmaf_rn(__uint_as_float(v[0]), f.x, a[0]);
                a[1] = __fmaf_rn(__uint_as_float(v[1]), f.y, a[1]);
                a[2] = __fmaf_rn(__uint_as_float(v[2]), f.z, a[2]);
                a[3] = __fmaf_rn(__uint_as_float(v[3]), f.w, a[3]);
              }
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[b]);
        it += blocks;
      }
      if (!ok) break;

      if constexpr (MODE == kFewDown) {
        // the expert's tokens, weighted, into the block's fp32 sums, eight in
        // flight.  The groups hold different tokens of one expert, but a token
        // may change groups from one expert to the next: each expert waits
        // for the last.
        if (C::kGroups > 1 && segs > 0 && !__all_sync(0xFFFFFFFFu, mbar_wait(seg_bar, (segs - 1) & 1u))) {
          expired();
          break;
        }
#pragma unroll
        for (int q = 0; q < C::kChunks; ++q) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int t0 = chunk0(q) + h * 8;
            if (t0 >= n) break;
            float* to[8];
            float w[8], old[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int at = pair0 + (t0 + i < n ? t0 + i : t0);
              to[i] = sAcc + sTok[at] * 128 + row;
              w[i] = sWt[at];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) old[i] = *to[i];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (t0 + i < n) *to[i] = __fmaf_rn(w[i], acc[q][0][h * 8 + i], old[i]);
          }
        }
        if (C::kGroups > 1) {
          __syncwarp();
          if (lane == 0) mbar_arrive(seg_bar);
        }
      } else {
        // a rolled loop over the meetings, so that the epilogue's code stays
        // small: it runs once per 128 columns, from a cold instruction cache
#pragma unroll 1
        for (int c = 0; c < kSubs && sub0(c) < n; ++c) {
          float x[C::kTiles][C::kRedTok];
#pragma unroll
          for (int cc = 0; cc < kSubs; ++cc)
            if (cc == c) {
#pragma unroll
              for (int t = 0; t < C::kTiles; ++t)
#pragma unroll
                for (int q = 0; q < C::kRedTok; ++q) x[t][q] = acc[(cc * C::kRedTok + q) / 16][t][(cc * C::kRedTok + q) % 16];
            }
          if (lgW > 0) meet(x, n - sub0(c));
          if (!ok) break;
          if constexpr (MODE == kFewLinear) {
            finish_rows(c, x[0]);
          } else {
            // h = silu(g) u in fp32, its 1x128 group (the 128 threads' rows)
            // quantized straight from fp32: no rounding to bf16 on the way.
            // Slots without a token are computed along and not stored.
            const int own = own_of(c, n);
            if (own > 0) {
              float* am = sAmax + (grp * 2 + (quants & 1u)) * 4 * C::kRedTok;
              float h[C::kRedTok];
#pragma unroll
              for (int k = 0; k < C::kRedTok; ++k) h[k] = times_sigmoid(x[0][k], x[0][k]) * x[1][k];
#pragma unroll
              for (int k = 0; k < C::kRedTok; ++k) {
                const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(h[k]) & 0x7FFFFFFFu);
                if (lane == 0) am[k * 4 + quad] = __uint_as_float(top);
              }
              __syncwarp();
              if (lane == 0) mbar_arrive(&amax_bar[grp]);
              if (!__all_sync(0xFFFFFFFFu, mbar_wait(&amax_bar[grp], quants & 1u))) {
                expired();
                break;
              }
              ++quants;
              const uint64_t r0 = static_cast<uint64_t>(pair0 + sub0(c) + who);
              FGFP8_DCHECK(r0 + ((own - 1) << lgW) < static_cast<uint64_t>(p.T) * p.topk && sg.j * 128 + row < p.I);
#pragma unroll
              for (int k = 0; k < C::kRedTok; ++k) {
                // magnitude bits compare like the values, and a NaN above all of them
                const uint4 m4 = *reinterpret_cast<const uint4*>(am + k * 4);
                float inv;
                const float scale = scale_of_f32(__uint_as_float(max(max(m4.x, m4.y), max(m4.z, m4.w))), p.fmt, inv);
                const uint8_t code = quant_f32(h[k], scale, inv);
                const uint64_t r = r0 + (static_cast<uint64_t>(k) << lgW);
                if (k < own) {
                  p.Hq[r * p.I + sg.j * 128 + row] = code;
                  if (row == 0) p.Hs[r * (p.I / 128) + sg.j] = scale;
                }
              }
            }
          }
        }
        if (!ok) break;
      }
      ++segs;
    }

    if constexpr (MODE == kFewDown) {
      // the block's sums over all experts, residual added, one rounding
      if (C::kGroups > 1 && ok && segs > 0 && !__all_sync(0xFFFFFFFFu, mbar_wait(seg_bar, (segs - 1) & 1u))) expired();
      if (C::kGroups > 1 && S > 1) {
        // Many tokens: all of them meet at once in the stages, which are free
        // when every rank has promoted its last block (eight at a time through
        // sRed took 8 us for 64 tokens): [rank][slot][128] in sA, token t to
        // rank t % S, slot t / S.
        float* ring = reinterpret_cast<float*>(sA);
        const int per = NT >> lgS;
        cluster_wait();                                              // the others' barriers exist
        if (ok && lane < S) mbar_arrive_cluster(map_to_rank(smem_u32(&red_empty[0]), lane));
        if (ok && !__all_sync(0xFFFFFFFFu, mbar_wait_cluster(&red_empty[0], 0))) expired();
        if (ok) {
#pragma unroll 4
          for (int t = grp; t < p.T; t += C::kGroups)
            st_cluster_f32(map_to_rank(smem_u32(ring + (rank * per + (t >> lgS)) * 128 + row), t & (S - 1)),
                           sAcc[t * 128 + row]);
          __syncwarp();
          if (lane < S) mbar_arrive_cluster(map_to_rank(smem_u32(&red_full[0]), lane));
          if (!__all_sync(0xFFFFFFFFu, mbar_wait_cluster(&red_full[0], 0))) expired();
        }
        meets = 1;
#pragma unroll 1
        for (int c = 0; c < kSubs && sub0(c) < p.T && ok; ++c) {
          float x[C::kRedTok];
#pragma unroll
          for (int k = 0; k < C::kRedTok; ++k) x[k] = 0.0f;
          const float* from = ring + (sub0(c) >> lgS) * 128 + row;
#pragma unroll 1
          for (int r = 0; r < S; ++r) {
#pragma unroll
            for (int k = 0; k < C::kRedTok / 2; ++k)                 // S >= 2
              if (k < slots) x[k] += from[(r * per + k) * 128];
          }
          finish_rows(c, x);
        }
      } else {
#pragma unroll 1
        for (int c = 0; c < kSubs && sub0(c) < p.T && ok; ++c) {
          float x[1][C::kRedTok];
#pragma unroll
          for (int q = 0; q < C::kRedTok; ++q) x[0][q] = sAcc[(sub0(c) + q) * 128 + row];
          if (S > 1) meet(x, p.T - sub0(c));
          if (!ok) break;
          finish_rows(c, x[0]);
        }
      }
    }
    if (S > 1 && meets == 0) cluster_wait();
  }

  // ---- teardown
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (S > 1) {                                    // no rank leaves while another may still write to it
    if (warp >= kTokWarp0) cluster_wait();        // (the first phase)
    cluster_arrive();
    cluster_wait();
  }
  if (warp == kMmaWarp) tmem_dealloc(tmem_base, C::kTmemCols);
}

}  // namespace fgfp8
