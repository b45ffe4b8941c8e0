// Backward pass over packed sequences with grouped heads, by recomputation, for
// sm_103a. The computation of one (128-key tile, 128-query tile) pair is that of
// fa_bwd.cu (five tcgen05 products, P and dS recomputed by two warpgroups, the
// dQ partial drained by a third and added into an fp32 accumulator with TMA
// reduce-add). What is different:
//   * a work item is a key tile of one (sequence, key/value head). A CTA loops
//     over the G query heads of that head and their live query tiles, so dK and
//     dV of a shared head are summed in TMEM, in a fixed order, and written
//     once; nothing of them is added through memory;
//   * where there are few items (few key/value heads, few tiles) they are cut into
//     parts, ranges of those (query head, query tile) steps, whose fp32 sums the
//     last pass adds up in order (packed_bwd_parts: forward and backward of 17
//     documents of 10-676 tokens, 7 / 1 heads, d = 80: 107 us whole, 49 in parts;
//     of three of 5-200, 8 / 2 heads, d = 64: 25.7 and 22.4);
//   * items come from a list made on the device, heaviest first, as in the
//     forward (fa_packed_fwd.cu);
//   * tiles are boxes of the strided [token, head, d] tensors and may run into
//     the next sequence: the MMA warp zeroes the rows past the end in shared
//     memory (K and V once per item, Q and dO at a head's last query tile)
//     before the products that read them, so what lies there (NaN included)
//     reaches no sum;
//   * the row statistics and the dQ accumulator are kept over sequences padded
//     to whole tiles, where the 128-row copies need no bounds;
//   * dK and dV go from registers to global memory (as O does in the forward), so
//     K and V of the next item load as soon as this one's last product has read
//     theirs, while dK and dV are written.
//
// Launches (after the plan, for more than kDirect sequences): the pre-pass
// (D = rowsum(dO * O), LSE * log2 e, zeroed accumulator; for scores of their own
// D = rowsum(P * dP), fa_packed_dots.cuh), the main kernel, and dQ = 16-bit(scale
// * accumulator).
//
// Scores of their own (SCORE): P = exp(u - LSE) of the capped and lowered scores
// u, and dS = P (dP - D) (1 - tanh^2), whose factor joins P in registers once P has
// been packed for dV. With a prefix, a key tile that begins in it has all query
// tiles of its sequence.
//
// Roundings: P and dS go to the inputs' 16-bit type for the products that read
// them (half a step each; dS is what the error of dQ and dK is made of: 2.5e-3 of
// their norm in bf16, where rounding them alone makes 1.7e-3); D, sums and
// accumulators are fp32.
//
// Bound: 10 d operations per visible pair; a step of five products takes 2.9 us
// at d = 128 where the tensor cores alone would take 1.7 (one S and one dP tile
// fit beside the accumulators, so P and dS of a tile stand between its products).
// Measured, bf16, causal, 32 / 8 heads, d = 128: two sequences of 4547 and 5127
// tokens 0.93 ms in the main kernel, 47 us pre-pass, 32 us dQ; 16 sequences of
// 32-977 tokens 167, 35 and 26 us (the passes around are at the bandwidth of the
// fp32 accumulator).
#pragma once

#include "fa_packed.cuh"
#include "fa_packed_dots.cuh"

#include <type_traits>

namespace fa {

namespace {

// Warp roles: 0-3 and 4-7 recompute P and dS for query columns 0-63 and 64-127
// (thread = key row), 8-11 drain dQ (thread = query row), 12 TMA producer,
// 13 MMA, 14-15 idle (their warpgroup hands its registers to the others).
constexpr int kGroups = 2;
constexpr int kCols = kTile / kGroups;
constexpr int kBwdThreads = 128 * (kGroups + 2);
constexpr int kDrainWarp0 = 4 * kGroups;
constexpr int kProducerWarp = kDrainWarp0 + 4;
constexpr int kMmaWarp = kProducerWarp + 1;
constexpr int kComputeRegs = 160, kDrainRegs = 96, kOtherRegs = 96;
static_assert(128 * (kGroups * kComputeRegs + kDrainRegs + kOtherRegs) == kBwdThreads * 128,
              "the reallocated registers must add up to the launch allocation");

template <int D>
struct PackedBwdLayout {
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kHalves = D / 64;
  static constexpr int kStages = (D == 64) ? 3 : 2;   // Q/dO ring depth (smem-limited at d = 128)
  static constexpr int kKV = (D == 64) ? 2 : 1;        // K/V buffers (a second one fits at d = 64)
  static constexpr int kKVBytes = 2 * kTileBytes;
  static constexpr int kK = 0;                                // [kKV] buffers of K then V
  static constexpr int kV = kK + kTileBytes;
  static constexpr int kQ = kKV * kKVBytes;                   // [stages]
  static constexpr int kdO = kQ + kStages * kTileBytes;       // [stages]
  static constexpr int kdS = kdO + kStages * kTileBytes;      // 128 x 128 bf16
  static constexpr int kRow = kdS + kTile * kTile * 2;        // [stages] x (LSE2[128], D[128])
  static constexpr int kBar = kRow + kStages * 2 * kTile * 4;
  static constexpr int bKV = 0;                            // [kKV]
  static constexpr int bQFull = bKV + kKV;
  static constexpr int bQEmpty = bQFull + kStages;
  static constexpr int bdOFull = bQEmpty + kStages;        // [stages]
  static constexpr int bdOFree = bdOFull + kStages;        // [stages]: dQ staging read by TMA (1 arrival, 4 per warp at d = 128)
  static constexpr int bSFull = bdOFree + kStages;
  static constexpr int bPFull = bSFull + 1;
  static constexpr int bdPFull = bPFull + 1;
  static constexpr int bdSFull = bdPFull + 1;
  static constexpr int bdSEmpty = bdSFull + 1;
  static constexpr int bdQFull = bdSEmpty + 1;
  static constexpr int bdQFree = bdQFull + 1;
  static constexpr int bFinal = bdQFree + 1;
  static constexpr int bDrain = bFinal + 1;
  static constexpr int bKVFree = bDrain + 1;   // [kKV]: the item's last product has read K and V
  // work items reach the other roles through a ring filled by the producer
  static constexpr int kItemRing = 4, kItemInts = 9;
  static constexpr int bItemFull = bKVFree + kKV;            // [kItemRing]
  static constexpr int bItemEmpty = bItemFull + kItemRing;   // [kItemRing]: MMA warp, compute and drain warps
  static constexpr int bdSHalf = bItemEmpty + kItemRing;     // the first 32 dS^T columns of each warpgroup
  static constexpr int bClc = bdSHalf + 1;                   // the next item's cancellation answer has arrived
  static constexpr int kNumBars = bClc + 1;
  static constexpr int kMisc = (kBar + 8 * kNumBars + 15) & ~15;   // tmem slot, abort flag, -, wait limit
  static constexpr int kRing = kMisc + 16;                    // [kItemRing] x {key tile, head, first row, length, first padded tile, steps, first query head, first query tile, place of a part}
  static constexpr int kClc = (kRing + 4 * kItemInts * kItemRing + 15) & ~15;   // 16-byte answer of a launch cancellation
  static constexpr int kSmemBytes = kClc + 16;
  // the dQ partial is drained per warp (each warp adds its own 32 rows) at
  // d = 128 and by the four warps together (whole 128-row boxes) at d = 64:
  // measured, each is the faster one at its width
  static constexpr bool kGroupDrain = (D == 64);
  static_assert(kSmemBytes <= 232448, "shared memory budget");
};

// First query tile that sees a key of tile kj: the first of all while the tile
// begins within the prefix.
template <bool PRE>
__device__ __forceinline__ int first_query_tile(bool causal, int kj, int prefix) {
  return causal && !(PRE && kTile * kj < prefix) ? kj : 0;
}

// P (log2 arguments in, 16-bit pairs out) and what of it stands in dS, of a key
// row against 64 queries: pk the pairs of P_c = 2^(u2_c - lse2_c), x_c = P_c times
// the cap's slope 1 - tanh^2. side: -1 where the queries' tile lies before the
// key's, 1 behind it, 0 the same; far: first query - key. Queries c < lim do not
// see the key (what they give, an infinity perhaps, is replaced).
template <int SCORE, bool F16, int kC>
__device__ __forceinline__ void score_p(float (&x)[kC], uint32_t (&pk)[kC / 2], const float* lse2, const ScoreParams& sp,
                                        float sl2, float slope2, float far, int side, bool masked, int lim) {
  const bool bias = sp.slopes != nullptr;
  const float sl = side > 0 ? -slope2 : slope2;
  // what is added to a pair's capped scores
  auto added = [&](int c) -> float2 {
    const float2 l = *reinterpret_cast<const float2*>(lse2 + c);
    float2 u = make_float2(-l.x, -l.y);
    if (bias) {
      float2 d = __fadd2_rn(make_float2(far, far), make_float2((float)c, (float)(c + 1)));
      if (side == 0) d = make_float2(-fabsf(d.x), -fabsf(d.y));
      u = __ffma2_rn(make_float2(sl, sl), d, u);
    }
    return u;
  };
  if constexpr (SCORE == kScoreCap) {
    // Without a bias, and all scores of the warp within the polynomial's limit: in one
    // piece, its products beside the exponentials. (One exponential and half a
    // reciprocal a score less: two sequences of 4547 and 5127 tokens, 32 / 8 heads,
    // d = 128, 1885 -> 1669 us with gradients.) A pair is two queries: a NaN score of one
    // stays out of the other's; where the one sees the key, its LSE is NaN and brings the
    // NaN back.
    float top[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < kC; c += 2) top[(c >> 1) & 3] = fmax3(top[(c >> 1) & 3], fabsf(x[c]), fabsf(x[c + 1]));
    const bool small = __all_sync(0xFFFFFFFFu, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) <= sp.limit);
    auto pair = [&](int c, float2 th, float2 f, float2 u) {
      u = __ffma2_rn(th, make_float2(sp.c2, sp.c2), u);
      const float2 p = make_float2(ex2(u.x), ex2(u.y));
      pk[c / 2] = pack2<F16>(p.x, p.y);
      const float2 y = __fmul2_rn(p, f);
      x[c] = y.x;
      x[c + 1] = y.y;
    };
    if (small && !bias) {
#pragma unroll
      for (int c = 0; c < kC; c += 2) {
        const float2 l = *reinterpret_cast<const float2*>(lse2 + c);
        const float2 th = tanh_small2(make_float2(x[c], x[c + 1]), sp);
        pair(c, th, __ffma2_rn(make_float2(-th.x, -th.y), th, make_float2(1.f, 1.f)), make_float2(-l.x, -l.y));
      }
    } else {
#pragma unroll
      for (int c = 0; c < kC; c += 2) {
        float2 f;
        const float2 th = tanh_slope2(make_float2(x[c], x[c + 1]), sp, f);
        pair(c, th, f, added(c));
      }
    }
  } else {
#pragma unroll
    for (int c = 0; c < kC; c += 2) {
      const float2 u = __ffma2_rn(make_float2(x[c], x[c + 1]), make_float2(sl2, sl2), added(c));
      x[c] = ex2(u.x);
      x[c + 1] = ex2(u.y);
      pk[c / 2] = pack2<F16>(x[c], x[c + 1]);
    }
  }
  if (masked)
#pragma unroll
    for (int c = 0; c < kC; ++c)
      if (c < lim) {
        x[c] = 0.f;
        pk[c / 2] &= (c & 1) ? 0x0000FFFFu : 0xFFFF0000u;
      }
}

template <int D, bool F16, int SLOTS, int SCORE>
__global__ void __launch_bounds__(kBwdThreads, 1)
fa_packed_bwd_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                     const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap tdo,
                     const __grid_constant__ CUtensorMap tdq, const PackedBwdParams p) {
  using L = PackedBwdLayout<D>;
  constexpr bool PRE = SCORE != kScorePlain;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);

  const int tid = threadIdx.x;
  // (from a shuffle, so that the compiler knows it to be the same in all lanes:
  // the operands of an MMA are uniform registers, and in a branch that it takes
  // for divergent each MMA costs some 40 instructions more)
  const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  const int lane = tid & 31;

  // An item: key tile kj of the sequence of rows start .. start + len - 1, for
  // key/value head hk; its query tiles i0 .. nT - 1 of each of the G query
  // heads, a head after the other, or `steps` of them from tile i of query head
  // hq on, whose sums go to tile `place` of the parts (dK; dV's Hk cap_tiles
  // behind); slot0 is the sequence's first padded tile.
  struct Item {
    int kj, hk, start, len, slot0, steps, hq, i, place;
    int i0, nT;
    int pre;   // PRE: keys that every query sees
    __device__ __forceinline__ int tail() const { return len & (kTile - 1); }
  };
  auto bar = [&](int i) -> uint32_t { return sbase + L::kBar + 8u * (uint32_t)i; };
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  volatile uint32_t* abort_flag = misc + 1;
  Ctl ctl{p.err, abort_flag};
  int* ring = reinterpret_cast<int*>(smem + L::kRing);
  // item k of this CTA from the ring; kj < 0 when none is left or a wait
  // failed (then ok is false too)
  auto take_item = [&](int k, bool& ok) -> Item {
    const int rs = k % L::kItemRing;
    const uint32_t ph = (uint32_t)(k / L::kItemRing) & 1u;
    ok = bar_wait_warp(bar(L::bItemFull + rs), ph, ctl, 355);
    Item w{-1, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
    if (!ok) return w;
    w.kj = __shfl_sync(0xFFFFFFFFu, ring[L::kItemInts * rs], 0);   // (the same in all lanes, as the compiler then knows)
    w.hk = __shfl_sync(0xFFFFFFFFu, ring[L::kItemInts * rs + 1], 0);
    w.start = __shfl_sync(0xFFFFFFFFu, ring[L::kItemInts * rs + 2], 0);
    w.len = __shfl_sync(0xFFFFFFFFu, ring[L::kItemInts * rs + 3], 0);
    w.slot0 = __shfl_sync(0xFFFFFFFFu, ring[L::kItemInts * rs + 4], 0);
    w.steps = __shfl_sync(0xFFFFFFFFu, ring[L::kItemInts * rs + 5], 0);
    w.hq = __shfl_sync(0xFFFFFFFFu, ring[L::kItemInts * rs + 6], 0);
    w.i = __shfl_sync(0xFFFFFFFFu, ring[L::kItemInts * rs + 7], 0);
    w.place = __shfl_sync(0xFFFFFFFFu, ring[L::kItemInts * rs + 8], 0);
    w.nT = (w.len + kTile - 1) / kTile;
    if constexpr (PRE)
      if (w.kj >= 0) {
        w.pre = prefix_of(w.kj);
        w.kj = tile_of(w.kj);
      }
    w.i0 = first_query_tile<PRE>(p.causal != 0, w.kj, w.pre);
    mbar_arrive_warp(bar(L::bItemEmpty + rs));
    return w;
  };

  if ((sbase & 1023u) != 0u) {   // uniform across the CTA: nothing has started yet
    if (tid == 0) {
      uint32_t dummy = 0;   // report_error writes only the abort flag
      Ctl c0{p.err, &dummy};
      report_error(c0, kErrSmemAlign, 350);
    }
    return;
  }

  if (tid == 0) {
    for (int i = 0; i < L::kNumBars; ++i)
      mbar_init(bar(i), (i == L::bPFull || i == L::bdSFull || i == L::bdSHalf) ? (uint32_t)(4 * kGroups)
                        : i == L::bdQFree ? 4u                                       // the four drain warps
                        : (!L::kGroupDrain && i >= L::bdOFree && i < L::bdOFree + L::kStages) ? 4u   // the drain warps
                        : (i >= L::bItemEmpty && i < L::bItemEmpty + L::kItemRing)
                            ? (uint32_t)(1 + 4 * kGroups + 4) : 1u);   // arrivals: MMA, compute and drain warps
    abort_flag[0] = 0u;
    abort_flag[2] = p.wait_us;   // the wait limit, read by the slow path of every wait
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(misc), 512);
    tmem_relinquish();
  }
  // global memory is read and written only from here on: what the pre-pass
  // wrote (row statistics, zeroed accumulator) is visible, and the plan
  grid_dep_wait();
  grid_dep_launch();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  const uint32_t tmem = misc[0];
  const uint32_t tdV = tmem;
  const uint32_t tdK = tmem + (uint32_t)D;
  const uint32_t tS = tmem + 2u * D;
  const uint32_t tP = tmem + 2u * D + 128u;   // dP^T (and at d = 128 then the dQ partial)
  // At d = 64 the dQ partial has 64 columns of its own (2d + 256 + d <= 512),
  // which allows a schedule where nothing waits for its drain (see the MMA
  // issuer); at d = 128 it reuses the dP^T columns.
  constexpr bool kOwnDQ = (D == 64);
  constexpr bool kSplitDS = (D == 128);   // dS^T handed to dK in two halves
  const uint32_t tQ = kOwnDQ ? tmem + 2u * D + 256u : tP;
  // S^T of the next tile right behind dV (before dK) at d = 64; at d = 128
  // behind dQ, which leaves its Q load the longest window
  constexpr bool kEarlyS = kOwnDQ;
  // dS^T for dK: packed over the consumed dP^T columns when the next S^T is
  // issued before dK (dQ, which reuses those columns at d = 128, is issued
  // after dK, and the tensor pipe runs in issue order), else into the S
  // columns next to P^T
  const uint32_t tDS = kEarlyS ? tP : tS + (uint32_t)(kCols / 2);
  // TMEM column of K step ks (16 queries) of the packed P^T / dS^T: each
  // warpgroup packs its kCols queries into the first kCols / 2 of its own
  // kCols S (or dP^T) columns
  auto packed_col = [](int ks) -> uint32_t {
    constexpr int kSteps = kCols / 16;   // K steps per warpgroup
    return (uint32_t)(kCols * (ks / kSteps) + 8 * (ks % kSteps));
  };

  // Every role walks the same items in the same order and counts the query
  // tiles it has passed over all of them (g): ring slots and barrier phases
  // follow g, so the pipeline runs on across item boundaries. Work items walk
  // groups of p.group key/value heads (whose Q, dO and dQ accumulator fit in L2
  // together), within a group the list's order (heaviest first), and for each
  // entry the heads of the group.
  const size_t Np = (size_t)p.cap_tiles * kTile;
  if (warp >= kProducerWarp) regs_dec<kOtherRegs>();
  if (warp == kProducerWarp) {
    // ------------------------------------------------------------ producer (warp-wide)
    if (lane == 0) {
      tma_prefetch_map(&tq);
      tma_prefetch_map(&tk);
      tma_prefetch_map(&tv);
      tma_prefetch_map(&tdo);
    }
    // up to kDirect sequences: the list is made here and items are taken by
    // cancelling CTAs of the grid that have not started; else both are the plan's
    const bool direct = p.B <= kDirect;
    DirectList<SLOTS, PRE> dl;
    int n_items = 0;
    if (direct) {
      dl.init(p.cu, p.score.prefix, p.B, p.total, kTile, p.cap_tiles, p.causal != 0, p.err);
      n_items = dl.items;
    } else {
      n_items = p.plan->items;
    }
    const int heads = p.Hk * p.parts, total = n_items * heads;
    int nq = 0, nd = 0, nkv = 0;
    bool clc_out = false;        // a cancellation answer is outstanding
    uint32_t clc = 0u;           // answers received
    bool ok = true;
    int g = 0;
    for (int k = 0; ok; ++k) {
      // claim the next item and hand it to the other roles
      const int rs = k % L::kItemRing;
      if (k >= L::kItemRing &&
          !(ok = bar_wait_warp(bar(L::bItemEmpty + rs), (uint32_t)(k / L::kItemRing - 1) & 1u, ctl, 354)))
        break;
      Item w{-1, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
      for (bool first = k == 0;; first = false) {
        int item = (int)blockIdx.x;
        if (!first && !direct) {
          item = (int)gridDim.x + __shfl_sync(0xFFFFFFFFu, lane == 0 ? (int)atomicAdd(&p.plan->sched, 1u) : 0, 0);
        } else if (!first) {
          if (lane == 0) {
            mbar_arrive_expect_tx(bar(L::bClc), 16u);
            clc_try_cancel(sbase + L::kClc, bar(L::bClc));
          }
          __syncwarp();
          clc_out = true;
          if (!(ok = bar_wait_warp(bar(L::bClc), clc & 1u, ctl, 356))) break;
          clc_out = false;
          ++clc;
          item = __shfl_sync(0xFFFFFFFFu, clc_first_ctaid_x(sbase + L::kClc), 0);
          if (item < 0) break;
          if (item >= total) continue;   // past the list: cancelled too, until none is left
        }
        if (item >= total) break;
        int hk = 0;
        const int idx = split_grouped(item, p.group, n_items, heads, &hk);
        PackedItem pi;
        if (direct) {
          pi = dl.at(idx, p.causal != 0);
          // causal: key tile kj has nT - kj query tiles, the list's c is one less
          if (p.causal) pi.c = (pi.len + kTile - 1) / kTile - 1 - pi.c;
          if constexpr (PRE) w.pre = dl.prefix;
        } else {
          pi = p.items[idx];
          if (pi.len <= 0) continue;     // left out by the plan
          if constexpr (PRE) {
            w.pre = __shfl_sync(0xFFFFFFFFu, prefix_of(pi.c), 0);
            pi.c = tile_of(pi.c);
          }
        }
        w.len = __shfl_sync(0xFFFFFFFFu, pi.len, 0);
        w.nT = (w.len + kTile - 1) / kTile;
        const int c = __shfl_sync(0xFFFFFFFFu, pi.c, 0);
        w.i0 = first_query_tile<PRE>(p.causal != 0, c, w.pre);
        w.start = __shfl_sync(0xFFFFFFFFu, pi.start, 0);
        w.slot0 = __shfl_sync(0xFFFFFFFFu, pi.slot0, 0);
        const int row = w.nT - w.i0, all = p.G * row;   // steps of the item, in query heads of `row`
        w.hk = hk;
        w.steps = all;
        w.hq = hk * p.G;
        w.i = w.i0;
        if (p.parts > 1) {
          const int part = hk % p.parts, parts = min(p.parts, all);
          if (part >= parts) continue;
          const int s0 = all * part / parts;
          w.steps = all * (part + 1) / parts - s0;
          w.hk = hk / p.parts;
          w.hq = w.hk * p.G + s0 / row;
          w.i += s0 % row;
          w.place = (part * 2 * p.Hk + w.hk) * p.cap_tiles + w.slot0 + c;
        }
        w.kj = c;
        break;
      }
      if (!ok) break;
      if (lane == 0) {
        ring[L::kItemInts * rs] = PRE && w.kj >= 0 ? with_prefix(w.kj, w.pre) : w.kj;
        ring[L::kItemInts * rs + 1] = w.hk;
        ring[L::kItemInts * rs + 2] = w.start;
        ring[L::kItemInts * rs + 3] = w.len;
        ring[L::kItemInts * rs + 4] = w.slot0;
        ring[L::kItemInts * rs + 5] = w.steps;
        ring[L::kItemInts * rs + 6] = w.hq;
        ring[L::kItemInts * rs + 7] = w.i;
        ring[L::kItemInts * rs + 8] = w.place;
        mbar_arrive(bar(L::bItemFull + rs));   // (release: the ring entry is visible to the waiters)
      }
      if (w.kj < 0) break;
      if (k >= L::kKV)   // K and V wait for the item before: into L2 until then
        for (int h = 0; h < L::kHalves; ++h) {
          tma_prefetch_3d_w(&tk, 64 * h, w.hk, w.start + kTile * w.kj);
          tma_prefetch_3d_w(&tv, 64 * h, w.hk, w.start + kTile * w.kj);
        }
#pragma unroll 1
      for (int it = 0, i = w.i, hq = w.hq; it < w.steps; ++it, ++g) {
        if (p.stall != 0u && g >= 1) { ok = false; break; }   // test of the timeout path: Q of tile 1 never comes
        const int s = g % L::kStages;
        const uint32_t n = (uint32_t)(g / L::kStages);
        // Q and the row statistics once dK has read the slot's Q; dO once the
        // dQ partial staged in the slot's dO buffer has been read
        if (g >= L::kStages && !(ok = bar_wait_warp(bar(L::bQEmpty + s), (n - 1) & 1u, ctl, 351))) break;
        mbar_arrive_expect_tx_w(bar(L::bQFull + s), L::kTileBytes + 2u * kTile * 4u);
        for (int h = 0; h < L::kHalves; ++h)
          tma_load_3d_w(sbase + L::kQ + s * L::kTileBytes + h * 16384, &tq, bar(L::bQFull + s), 64 * h, hq,
                        w.start + kTile * i);
        const size_t roff = (size_t)hq * Np + (size_t)kTile * (w.slot0 + i);
        bulk_load_w(sbase + L::kRow + s * 1024, p.lse2 + roff, kTile * 4, bar(L::bQFull + s));
        bulk_load_w(sbase + L::kRow + s * 1024 + 512, p.delta + roff, kTile * 4, bar(L::bQFull + s));
        ++nq;
        if (g >= L::kStages && !(ok = bar_wait_warp(bar(L::bdOFree + s), (n - 1) & 1u, ctl, 352))) break;
        mbar_arrive_expect_tx_w(bar(L::bdOFull + s), L::kTileBytes);
        for (int h = 0; h < L::kHalves; ++h)
          tma_load_3d_w(sbase + L::kdO + s * L::kTileBytes + h * 16384, &tdo, bar(L::bdOFull + s), 64 * h, hq,
                        w.start + kTile * i);
        ++nd;
        // K and V behind the first query tile of the item, whose loads only
        // wait for ring slots of the previous item: into buffer k % kKV, once the
        // last product of the item that used it before has read it
        if (it == 0) {
          const int kb = k % L::kKV;
          if (k >= L::kKV && !(ok = bar_wait_warp(bar(L::bKVFree + kb), (uint32_t)(k / L::kKV - 1) & 1u, ctl, 353))) break;
          mbar_arrive_expect_tx_w(bar(L::bKV + kb), 2u * L::kTileBytes);
          for (int h = 0; h < L::kHalves; ++h) {
            tma_load_3d_w(sbase + L::kK + kb * L::kKVBytes + h * 16384, &tk, bar(L::bKV + kb), 64 * h, w.hk,
                          w.start + kTile * w.kj);
            tma_load_3d_w(sbase + L::kV + kb * L::kKVBytes + h * 16384, &tv, bar(L::bKV + kb), 64 * h, w.hk,
                          w.start + kTile * w.kj);
          }
          ++nkv;
        }
        if (++i == w.nT) {
          i = w.i0;
          ++hq;
        }
      }
    }
    // every load and cancellation request issued has completed before the CTA exits
    if (lane == 0) {
      if (clc_out) drain_wait(bar(L::bClc), clc & 1u);
#pragma unroll 1
      for (int kb = 0; kb < L::kKV && kb < nkv; ++kb)
        drain_wait(bar(L::bKV + kb), (uint32_t)((nkv - 1 - kb) / L::kKV) & 1u);
#pragma unroll 1
      for (int s = 0; s < L::kStages; ++s) {
        if (s < nq) drain_wait(bar(L::bQFull + s), (uint32_t)((nq - 1 - s) / L::kStages) & 1u);
        if (s < nd) drain_wait(bar(L::bdOFull + s), (uint32_t)((nd - 1 - s) / L::kStages) & 1u);
      }
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issuer
    // the whole warp runs the schedule and one elected lane issues each MMA and
    // commit; all lanes take part when the rows past a sequence are zeroed
    {
      constexpr uint32_t idSP = idesc_16<F16>(128, 128, false, false);
      constexpr uint32_t idV = idesc_16<F16>(128, D, false, true);
      constexpr uint32_t idK = idesc_16<F16>(128, D, false, true);
      constexpr uint32_t idQ = idesc_16<F16>(128, D, true, true);
      const uint32_t dS0 = desc_lo(desc_mnmajor(sbase + L::kdS, 0));
      bool ok = true;
      int g = 0;
      // Shared-memory descriptors are a base's low word plus a constant step per
      // K step (mma_ss_lo).
      // S^T = K Q^T of running query tile g1 (tail: its first row past the
      // sequence, or 0)
      auto issue_s = [&](uint32_t sK, int g1, int tail) -> bool {
        const int s1 = g1 % L::kStages;
        if (!bar_wait_warp(bar(L::bQFull + s1), (uint32_t)(g1 / L::kStages) & 1u, ctl, 364)) return false;
        if (tail != 0) zero_tail_rows<D>(smem + L::kQ + s1 * L::kTileBytes, tail);
        tc_fence_after();
        const uint32_t dK0 = desc_lo(desc_kmajor(sK, 0)), dQ0 = desc_lo(desc_kmajor(sbase + L::kQ + s1 * L::kTileBytes, 0));
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          mma_ss_lo(tS, dK0 + (uint32_t)kmajor_step(ks), dQ0 + (uint32_t)kmajor_step(ks), idSP, ks > 0 ? 1u : 0u);
        mma_commit_w(bar(L::bSFull));
        return true;
      };
      for (int k = 0; ok; ++k) {
        const Item w = take_item(k, ok);
        if (w.kj < 0) break;
        int i = w.i;
        const int tail = w.tail(), steps = w.steps;
        const int kb = k % L::kKV;
        const uint32_t sK = sbase + L::kK + kb * L::kKVBytes, sV = sbase + L::kV + kb * L::kKVBytes;
        const uint32_t mK = desc_lo(desc_mnmajor(sK, 0));
        if (!(ok = bar_wait_warp(bar(L::bKV + kb), (uint32_t)(k / L::kKV) & 1u, ctl, 360))) break;
        if (tail != 0 && w.kj == w.nT - 1) {
          zero_tail_rows<D>(smem + L::kK + kb * L::kKVBytes, tail);
          zero_tail_rows<D>(smem + L::kV + kb * L::kKVBytes, tail);
        }
        if (!(ok = issue_s(sK, g, i == w.nT - 1 ? tail : 0))) break;
        for (int it = 0; it < steps; ++it, ++g) {
          const bool more = it + 1 < steps;
          const int inext = i + 1 < w.nT ? i + 1 : w.i0;
          const int tail_next = inext == w.nT - 1 ? tail : 0;
          const int s = g % L::kStages;
          const uint32_t sQ = sbase + L::kQ + s * L::kTileBytes;
          const uint32_t sdO = sbase + L::kdO + s * L::kTileBytes;
          // dP^T = V dO^T (at d = 128 the dQ partial of the previous tile must
          // have been read out of these columns)
          if (!kOwnDQ && g > 0 && !(ok = bar_wait_warp(bar(L::bdQFree), (uint32_t)(g - 1) & 1u, ctl, 362))) break;
          if (!(ok = bar_wait_warp(bar(L::bdOFull + s), (uint32_t)(g / L::kStages) & 1u, ctl, 366))) break;
          if (tail != 0 && i == w.nT - 1) zero_tail_rows<D>(smem + L::kdO + s * L::kTileBytes, tail);
          tc_fence_after();
          const uint32_t kdV = desc_lo(desc_kmajor(sV, 0)), kdO = desc_lo(desc_kmajor(sdO, 0));
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            mma_ss_lo(tP, kdV + (uint32_t)kmajor_step(ks), kdO + (uint32_t)kmajor_step(ks), idSP, ks > 0 ? 1u : 0u);
          mma_commit_w(bar(L::bdPFull));
          // dV += P^T dO (at it == 0 over the previous item's dV and dK, which
          // the compute warps have read out of TMEM before arriving on this P)
          if (!(ok = bar_wait_warp(bar(L::bPFull), (uint32_t)g & 1u, ctl, 363))) break;
          tc_fence_after();
          const uint32_t mdO = desc_lo(desc_mnmajor(sdO, 0));
#pragma unroll
          for (int ks = 0; ks < kTile / 16; ++ks)
            // P of each warpgroup's queries packed in the first half of its own S columns
            mma_ts_lo(tdV, tS + packed_col(ks), mdO + (uint32_t)mnmajor_step(ks), idV,
                   (it > 0 || ks > 0) ? 1u : 0u);
          // next S^T of this item: early, right behind dV (the tensor pipe
          // runs in issue order, so dV has read P first), so that P of the
          // next tile is recomputed while dK, dQ and the next dP run; else
          // after dQ, which leaves the next Q load the longest window
          if (kEarlyS && more && !(ok = issue_s(sK, g + 1, tail_next))) break;
          // dK += dS^T Q ; dQ_i = dS K. dS^T is packed like P (packed_col) from
          // tDS on; at d = 128 each warpgroup hands over its first 32 queries
          // (K steps 0, 1 and 4, 5) before the rest (2, 3 and 6, 7), so half of
          // dK runs while dS is finished
          const uint32_t mQ = desc_lo(desc_mnmajor(sQ, 0));
          // dQ_i = dS K: with dS^T handed over in halves, dQ goes right after
          // dS is complete, in front of the second half of dK, so that its
          // drain overlaps that half
          auto issue_dq = [&]() {
#pragma unroll
            for (int ks = 0; ks < kTile / 16; ++ks)
              mma_ss_lo(tQ, dS0 + (uint32_t)mnmajor_step(ks), mK + (uint32_t)mnmajor_step(ks), idQ, ks > 0 ? 1u : 0u);
            mma_commit_w(bar(L::bdQFull));
          };
#pragma unroll
          for (int half = kSplitDS ? 0 : 1; half < 2; ++half) {
            if (!(ok = bar_wait_warp(bar(half == 0 ? L::bdSHalf : L::bdSFull), (uint32_t)g & 1u, ctl, 365)))
              break;
            tc_fence_after();
            if (kSplitDS && half == 1) issue_dq();
#pragma unroll
            for (int k4 = 0; k4 < (kSplitDS ? 4 : 8); ++k4) {
              const int ks = kSplitDS ? 2 * half + (k4 & 1) + 4 * (k4 >> 1) : k4;
              mma_ts_lo(tdK, tDS + packed_col(ks), mQ + (uint32_t)mnmajor_step(ks), idK,
                           (it > 0 || ks > 0) ? 1u : 0u);
            }
          }
          if (!ok) break;
          mma_commit_w(bar(L::bQEmpty + s));   // the slot's Q has been read for the last time
          if (!kSplitDS) {
            // at d = 64 the previous dQ partial must have been read out of its columns
            if (kOwnDQ && g > 0 && !(ok = bar_wait_warp(bar(L::bdQFree), (uint32_t)(g - 1) & 1u, ctl, 362))) break;
            tc_fence_after();
            issue_dq();
          }
          mma_commit_w(bar(L::bdSEmpty));      // dK and dQ have read dS
          if (!kEarlyS && more && !(ok = issue_s(sK, g + 1, tail_next))) break;
          i = inext;
        }
        if (ok) {
          mma_commit_w(bar(L::bFinal));          // dV and dK of the item are complete
          mma_commit_w(bar(L::bKVFree + kb));    // and K and V may be loaded over
        }
      }
      mma_commit_w(bar(L::bDrain));
      drain_wait(bar(L::bDrain), 0);
    }
  } else if (warp < kDrainWarp0) {
    // ------------------------------------------------------------ P and dS (thread = key row)
    // warpgroup cw handles query columns kC cw .. kC cw + kC - 1 of each tile
    regs_inc<kComputeRegs>();
    constexpr int kC = kCols;
    const int cw = warp >> 2;
    const int cb = kC * cw;
    const int r = tid & 127;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const float sl2 = p.scale_log2;
    bool ok = true;
    int g = 0, nf = 0;
    [[maybe_unused]] int hq = 0, slope_of = -1;   // SCORE: the step's query head, and whose slope is held
    [[maybe_unused]] float slope2 = 0.f;
    for (int k = 0; ok; ++k) {
      const Item w = take_item(k, ok);
      if (!ok || w.kj < 0) break;
      const int krow = kTile * w.kj + r;
      hq = w.hq - 1;
      for (int it = 0, i = w.i; it < w.steps; ++it, ++g, i = i + 1 < w.nT ? i + 1 : w.i0) {
        const bool partial = PRE ? (p.causal && i <= w.kj && (w.kj + 1) * kTile > w.pre) || (w.kj + 1) * kTile > w.len
                                 : (p.causal && i == w.kj) || (w.kj + 1) * kTile > w.len;
        if constexpr (PRE) {
          if (it == 0 || i == w.i0) ++hq;
          if (p.score.slopes != nullptr && hq != slope_of) {
            slope2 = p.score.slopes[hq] * 1.4426950408889634f;
            slope_of = hq;
          }
        }
        const int s = g % L::kStages;
        if (!(ok = bar_wait_warp(bar(L::bQFull + s), (uint32_t)(g / L::kStages) & 1u, ctl, 370))) break;
        if (!(ok = bar_wait_warp(bar(L::bSFull), (uint32_t)g & 1u, ctl, 371))) break;
        tc_fence_after();
        const float* lse2 = reinterpret_cast<const float*>(smem + L::kRow + s * 1024) + cb;
        const float* dlt = lse2 + kTile;
        float x[kC];
        {
          uint32_t u0[32], u1[32];
          tmem_ld32(tS + lane_off + (uint32_t)cb, u0);
          tmem_ld32(tS + lane_off + (uint32_t)cb + 32u, u1);
          tmem_ld_wait(u0);
          tmem_ld_wait(u1);
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            x[c] = __uint_as_float(u0[c]);
            x[32 + c] = __uint_as_float(u1[c]);
          }
        }
        // the dV operand is P packed two queries per TMEM column into the first
        // half of this warpgroup's own S columns (the other warpgroup may still
        // be reading its half)
        if constexpr (SCORE == kScorePlain) {
          // P^T row: p[c] = exp2(s * scale * log2e - LSE2[query c])
#pragma unroll
          for (int c4 = 0; c4 < kC / 4; ++c4) {
            const float4 l = reinterpret_cast<const float4*>(lse2)[c4];   // one broadcast load per 4 queries
            x[4 * c4] = ex2(fmaf(x[4 * c4], sl2, -l.x));
            x[4 * c4 + 1] = ex2(fmaf(x[4 * c4 + 1], sl2, -l.y));
            x[4 * c4 + 2] = ex2(fmaf(x[4 * c4 + 2], sl2, -l.z));
            x[4 * c4 + 3] = ex2(fmaf(x[4 * c4 + 3], sl2, -l.w));
          }
          if (partial) {
            // key row krow is masked for query q0 + c when it lies past the
            // query (causal: c < krow - q0) or at or past the key length (every c)
            const int lim = krow >= w.len ? kC : (p.causal ? krow - (kTile * i + cb) : 0);
#pragma unroll
            for (int c = 0; c < kC; ++c)
              if (c < lim) x[c] = 0.f;
          }
          uint32_t pk[kC / 2];
#pragma unroll
          for (int c = 0; c < kC / 2; ++c) pk[c] = pack2<F16>(x[2 * c], x[2 * c + 1]);
          tmem_st32(tS + lane_off + (uint32_t)cb, pk);
        } else {
          // key row krow is masked for query q when it lies past the query (causal)
          // and past the prefix, or at or past the key length
          const int far = kTile * i + cb - krow;
          const int lim = krow >= w.len ? kC : (p.causal && krow >= w.pre ? -far : 0);
          uint32_t pk[kC / 2];
          score_p<SCORE, F16>(x, pk, lse2, p.score, sl2, slope2, (float)far, i < w.kj ? -1 : i > w.kj ? 1 : 0, partial, lim);
          tmem_st32(tS + lane_off + (uint32_t)cb, pk);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive_warp(bar(L::bPFull));

        // dS^T row: ds[c] = p[c] * (dP[c] - D[query c]) -> 16-bit -> swizzled smem
        if (!(ok = bar_wait_warp(bar(L::bdPFull), (uint32_t)g & 1u, ctl, 372))) break;
        if (g > 0 && !(ok = bar_wait_warp(bar(L::bdSEmpty), (uint32_t)(g - 1) & 1u, ctl, 373))) break;
        tc_fence_after();
        // at d = 128 both 32-column halves of this warpgroup's dP^T are loaded
        // before the first wait, so their TMEM latencies overlap (at d = 64 the
        // 32 extra live registers would spill)
        constexpr bool kBothHalves = (D == 128);
        uint32_t ud[kC / 32][32];
        if constexpr (kBothHalves) {
#pragma unroll
          for (int cc = 0; cc < kC / 32; ++cc) tmem_ld32(tP + lane_off + (uint32_t)cb + 32u * cc, ud[cc]);
#pragma unroll
          for (int cc = 0; cc < kC / 32; ++cc) tmem_ld_wait(ud[cc]);
        }
#pragma unroll
        for (int cc = 0; cc < kC / 32; ++cc) {
          if constexpr (!kBothHalves) {
            tmem_ld32(tP + lane_off + (uint32_t)cb + 32u * cc, ud[cc]);
            tmem_ld_wait(ud[cc]);
          }
          const uint32_t* u = ud[cc];
          uint32_t pk[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const int c0 = 32 * cc + 2 * c;
            const float g0 = __uint_as_float(u[2 * c]), g1 = __uint_as_float(u[2 * c + 1]);
            const float2 dl = reinterpret_cast<const float2*>(dlt)[c0 >> 1];
            const float d0 = x[c0] * (g0 - dl.x), d1 = x[c0 + 1] * (g1 - dl.y);
            pk[c] = pack2<F16>(d0, d1);
          }
          // dS^T also goes to TMEM (the A operand of dK), packed (tDS): over
          // this warpgroup's dP columns, which it has already read, or into the
          // second half of its S columns, after its P
          tmem_st16(tDS + lane_off + (uint32_t)cb + 16u * cc, pk);
#pragma unroll
          for (int k4 = 0; k4 < 4; ++k4) {
            uint8_t* dst = smem + L::kdS + tile_chunk(r, (cb >> 3) + 4 * cc + k4);
            *reinterpret_cast<uint4*>(dst) =
                make_uint4(pk[4 * k4], pk[4 * k4 + 1], pk[4 * k4 + 2], pk[4 * k4 + 3]);
          }
          if (kSplitDS && cc == 0) {   // the first 32 queries' dS^T is in TMEM: dK may start on them
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive_warp(bar(L::bdSHalf));
          }
        }
        tmem_st_wait();
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive_warp(bar(L::bdSFull));
      }

      // epilogue: the first warpgroup writes dV, the second scale * dK, from
      // registers: a lane holds 32 columns of its row at a time, as four 16-byte
      // chunks; transposed across its quad it holds one chunk of four rows, and a
      // quad writes 64 bytes of each, up to the sequence's end
      if (!ok || !(ok = bar_wait_warp(bar(L::bFinal), (uint32_t)nf & 1u, ctl, 375))) break;
      ++nf;
      tc_fence_after();
      const bool is_v = cw == 0;
      const uint32_t tacc = (is_v ? tdV : tdK) + lane_off;
      if (p.parts > 1) {
        // a part: fp32 sums into its own place, each thread its row (past the
        // sequence's end too: the tile is the item's own, and those are not read)
        float* part = p.part + ((size_t)kTile * (w.place + (is_v ? p.Hk * p.cap_tiles : 0)) + r) * p.d;
#pragma unroll 1
        for (int cc = 0; cc < D / 32; ++cc) {
          uint32_t u[32];
          tmem_ld32(tacc + 32u * cc, u);
          tmem_ld_wait(u);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (32 * cc + 4 * j < p.d)
              *reinterpret_cast<uint4*>(part + 32 * cc + 4 * j) =
                  make_uint4(u[4 * j], u[4 * j + 1], u[4 * j + 2], u[4 * j + 3]);
        }
        tc_fence_before();
        continue;
      }
      const float mul = is_v ? 1.f : p.scale;
      const int s4 = lane & 3;
      const int row0 = kTile * w.kj + 32 * (warp & 3) + (lane & ~3);   // the quad's first row
      const int64_t tok = is_v ? p.dv_tok : p.dk_tok;
      uint16_t* op = (is_v ? p.dv : p.dk) + (int64_t)(w.start + row0) * tok + w.hk * (is_v ? p.dv_head : p.dk_head) + 8 * s4;
#pragma unroll 1
      for (int cc = 0; cc < D / 32; ++cc) {
        uint32_t u[32];
        tmem_ld32(tacc + 32u * cc, u);
        tmem_ld_wait(u);
        uint32_t y[4][4];   // [word of a chunk][chunk of this row, then row of the quad]
#pragma unroll
        for (int wd = 0; wd < 4; ++wd) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            y[wd][j] = pack2<F16>(__uint_as_float(u[8 * j + 2 * wd]) * mul, __uint_as_float(u[8 * j + 2 * wd + 1]) * mul);
          quad_transpose(y[wd], (uint32_t)s4);
        }
        if (32 * cc + 8 * s4 < p.d) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (row0 + j < w.len)
              *reinterpret_cast<uint4*>(op + j * tok + 32 * cc) = make_uint4(y[0][j], y[1][j], y[2][j], y[3][j]);
        }
      }
      tc_fence_before();   // (the next item's first dV waits for this warp's next P)
    }
  } else if (warp < kProducerWarp) {
    // ------------------------------------------------------------ dQ drain (thread = query row)
    // TMEM -> fp32 rows staged in this iteration's dO ring slot (dead once dQ
    // has completed) in two rounds of 32-column boxes, 128-byte swizzled ->
    // TMA reduce-add into the accumulator. The TMEM columns are released as
    // soon as they are all in registers or staged; the slot goes back to the
    // producer when its last round has been read.
    //   d = 128: each warp stages and adds its own 32 query rows (boxes of 32
    //            rows) and synchronises only within itself.
    //   d = 64:  the four warps stage whole 128-row boxes that one thread adds,
    //            meeting at named barriers; after each wait that one of them
    //            may fail they agree with group_all, so that they always take
    //            the same branch and none waits at a barrier another has left.
    regs_dec<kDrainRegs>();
    constexpr uint32_t kDrainBar = 1u + kGroups;   // named barrier of the drain warps (d = 64)
    constexpr int kBoxesPerRound = L::kTileBytes / 16384;    // 1 (d = 64) or 2 (d = 128)
    constexpr int kRounds = D / 32 / kBoxesPerRound;
    const int r = tid - 32 * kDrainWarp0;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t sw = (uint32_t)((r >> 3) * 1024 + (r & 7) * 128);
    const uint32_t wrow = L::kGroupDrain ? 0u : 4096u * (uint32_t)(warp & 3);   // this warp's rows in a box
    bool ok = true;
    int g = 0;
    for (int k = 0; ok; ++k) {
      const Item w = take_item(k, ok);
      if constexpr (L::kGroupDrain) ok = group_all(kDrainBar, 128, ok);
      if (!ok || w.kj < 0) break;
      for (int it = 0, i = w.i, hq = w.hq; it < w.steps; ++it, ++g) {
        const int s = g % L::kStages;
        const uint32_t stage = (uint32_t)(L::kdO + s * L::kTileBytes);
        ok = bar_wait_warp(bar(L::bdQFull), (uint32_t)g & 1u, ctl, 380);
        if constexpr (L::kGroupDrain) ok = group_all(kDrainBar, 128, ok);
        if (!ok) break;
        tc_fence_after();
        uint32_t u[kBoxesPerRound][32];
#pragma unroll
        for (int b = 0; b < kBoxesPerRound; ++b) tmem_ld32(tQ + lane_off + 32u * b, u[b]);
#pragma unroll
        for (int b = 0; b < kBoxesPerRound; ++b) tmem_ld_wait(u[b]);
#pragma unroll
        for (int round = 0; round < kRounds; ++round) {
          if (round == kRounds - 1) {
            tc_fence_before();
            mbar_arrive_warp(bar(L::bdQFree));   // every dQ column is in registers or staged
          }
          if (round > 0) {              // the previous round has been read out of the slot
            if constexpr (L::kGroupDrain) {
              if (r == 0) bulk_wait_group_read_all();
              named_bar_sync(kDrainBar, 128);
            } else {
              if (lane == 0) bulk_wait_group_read_all();
              __syncwarp();
            }
          }
#pragma unroll
          for (int b = 0; b < kBoxesPerRound; ++b)
#pragma unroll
            for (int k8 = 0; k8 < 8; ++k8) {    // 8 chunks of 4 fp32 per 32-column box
              const uint32_t o = sw + (uint32_t)((k8 ^ (r & 7)) << 4);
              *reinterpret_cast<uint4*>(smem + stage + 16384 * b + o) =
                  make_uint4(u[b][4 * k8], u[b][4 * k8 + 1], u[b][4 * k8 + 2], u[b][4 * k8 + 3]);
            }
          fence_proxy_async_smem();
          if constexpr (L::kGroupDrain)
            named_bar_sync(kDrainBar, 128);
          else
            __syncwarp();
          if (L::kGroupDrain ? r == 0 : lane == 0) {
            const int row0 = kTile * (w.slot0 + i) + (L::kGroupDrain ? 0 : 32 * (warp & 3));
#pragma unroll
            for (int b = 0; b < kBoxesPerRound; ++b)
              if (32 * (round * kBoxesPerRound + b) < p.d)   // boxes wholly past the head dimension hold zeros
                tma_reduce_add_3d(&tdq, sbase + stage + 16384u * b + wrow, 32 * (round * kBoxesPerRound + b),
                                  row0, hq);
            bulk_commit_group();
          }
          if (round + 1 < kRounds) {    // the next columns into registers while the round is read
#pragma unroll
            for (int b = 0; b < kBoxesPerRound; ++b)
              tmem_ld32(tQ + lane_off + 32u * ((round + 1) * kBoxesPerRound + b), u[b]);
#pragma unroll
            for (int b = 0; b < kBoxesPerRound; ++b) tmem_ld_wait(u[b]);
          }
        }
        if (L::kGroupDrain ? r == 0 : lane == 0) {
          bulk_wait_group_read_all();
          mbar_arrive(bar(L::bdOFree + s));
        }
        if (++i == w.nT) {
          i = w.i0;
          ++hq;
        }
      }
    }
    if (L::kGroupDrain ? r == 0 : lane == 0) bulk_wait_group_all();     // reductions complete before exit
  }

  tc_fence_before();
  __syncthreads();
  if (tid == 0) report_aborted(ctl);
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Padded tile `tile`, from a list of SLOTS sequences a lane or (0) the plan's; len 0 where there is none (whole warps call it together).
// PRE (lists of a lane only): its sequence's prefix too.
template <int SLOTS, bool PRE = false>
__device__ __forceinline__ PackedItem padded_tile(const PackedBwdParams& p, int tile, int* prefix = nullptr) {
  if constexpr (SLOTS > 0) {
    DirectList<SLOTS, PRE> dl;
    dl.read(p.cu, p.score.prefix, p.B, p.total, kTile, p.cap_tiles, nullptr);
    const PackedItem it = dl.unit(tile);
    if constexpr (PRE) *prefix = dl.prefix;
    return it;
  }
  if (tile >= p.plan->tiles) return PackedItem{0, 0, 0, 0};
  PackedItem it = p.tiles[tile];
  it.c = tile_of(it.c);   // (its prefix lies above)
  // (a sequence past the padded rows, of bounds that overlap, is left out)
  return it.slot0 + (it.len + kTile - 1) / kTile > p.cap_tiles ? PackedItem{0, 0, 0, 0} : it;
}

// Per padded tile and query head: D = rowsum(dO * O) and LSE * log2(e) of its
// rows (0 and +inf past the sequence), and the dQ accumulator's tile zeroed.
// LANES neighbouring threads take a row, 8 columns each.
template <int LANES, bool F16, int SLOTS>
__global__ void __launch_bounds__(256) packed_bwd_pre_kernel(const PackedBwdParams p) {
  grid_dep_launch();
  const int tile = (int)(blockIdx.x / (unsigned)p.Hq), h = (int)(blockIdx.x % (unsigned)p.Hq);
  const PackedItem it = padded_tile<SLOTS>(p, tile);
  if (it.len == 0) return;
  const size_t row_off = ((size_t)h * p.cap_tiles + tile) * kTile;
  const int part = (int)threadIdx.x % LANES;
  const bool cols = 8 * part < p.d;
  for (int r = (int)threadIdx.x / LANES; r < kTile; r += 256 / LANES) {
    const int n = kTile * it.c + r;       // token of the sequence
    float acc = 0.f;
    if (n < it.len && cols) {
      const int64_t t = (int64_t)it.start + n;
      const uint4 a = *reinterpret_cast<const uint4*>(p.o + t * p.o_tok + h * p.o_head + 8 * part);
      const uint4 g = *reinterpret_cast<const uint4*>(p.dout + t * p.do_tok + h * p.do_head + 8 * part);
      const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, gw[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 af = unpack2<F16>(aw[k]);
        const float2 gf = unpack2<F16>(gw[k]);
        acc = fmaf(af.x, gf.x, acc);
        acc = fmaf(af.y, gf.y, acc);
      }
    }
#pragma unroll
    for (int off = LANES / 2; off > 0; off >>= 1) acc += __shfl_xor_sync(0xFFFFFFFFu, acc, off);
    // (rows past the sequence are added to as well, and never read)
    if (n < it.len && cols) {
      float4* z = reinterpret_cast<float4*>(p.dq_acc + (row_off + r) * p.d + 8 * part);
      z[0] = make_float4(0.f, 0.f, 0.f, 0.f);
      z[1] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (part == 0) {
      p.delta[row_off + r] = acc;
      p.lse2[row_off + r] =
          n < it.len ? p.lse[(size_t)h * p.total + it.start + n] * 1.4426950408889634f : INFINITY;
    }
  }
}

// dQ = 16-bit(scale * accumulator), one thread per 8 columns of a row. With
// items in parts (PARTS), blocks behind those sum the parts of dK and dV, kSumRows rows
// of a tile each, in the order of the parts.
constexpr int kSumRows = 32;

template <bool F16, bool PARTS, int SLOTS, bool PRE>
__global__ void __launch_bounds__(256) packed_bwd_dq_kernel(const PackedBwdParams p) {
  grid_dep_launch();
  const int parts = p.d / 8;
  auto put = [](uint16_t* dst, const float4& a, const float4& c, float mul) {
    *reinterpret_cast<uint4*>(dst) = make_uint4(pack2<F16>(a.x * mul, a.y * mul), pack2<F16>(a.z * mul, a.w * mul),
                                                pack2<F16>(c.x * mul, c.y * mul), pack2<F16>(c.z * mul, c.w * mul));
  };
  const unsigned n_dq = (unsigned)p.cap_tiles * (unsigned)p.Hq;
  if (!PARTS || blockIdx.x < n_dq) {
    const int tile = (int)(blockIdx.x / (unsigned)p.Hq), h = (int)(blockIdx.x % (unsigned)p.Hq);
    const PackedItem it = padded_tile<SLOTS>(p, tile);
    if (it.len == 0) return;
    const size_t row_off = ((size_t)h * p.cap_tiles + tile) * kTile;
    const int rows = min(kTile, it.len - kTile * it.c);
    for (int i = (int)threadIdx.x; i < rows * parts; i += 256) {
      const int r = i / parts, part = i % parts;
      const float4* src = reinterpret_cast<const float4*>(p.dq_acc + (row_off + r) * p.d + 8 * part);
      const int64_t t = (int64_t)it.start + kTile * it.c + r;
      put(p.dq + t * p.dq_tok + h * p.dq_head + 8 * part, src[0], src[1], p.scale);
    }
    return;
  }
  if constexpr (!PARTS) return;
  unsigned x = blockIdx.x - n_dq;
  const int first = kSumRows * (int)(x % (kTile / kSumRows));
  x /= kTile / kSumRows;
  const bool is_v = x % 2 != 0;
  x /= 2;
  const int hk = (int)(x % (unsigned)p.Hk), tile = (int)(x / (unsigned)p.Hk);
  int prefix = 0;
  const PackedItem it = padded_tile<SLOTS, PRE>(p, tile, &prefix);
  const int rows = min(kSumRows, it.len - kTile * it.c - first);
  if (it.len == 0 || rows <= 0) return;
  const int nT = (it.len + kTile - 1) / kTile;
  const int n = min(p.parts, p.G * (nT - first_query_tile<PRE>(p.causal != 0, it.c, prefix)));   // parts with steps
  const size_t head = (size_t)p.cap_tiles * kTile * p.d, step = 2 * p.Hk * head;
  const float* base = p.part + ((is_v ? p.Hk : 0) + hk) * head + ((size_t)tile * kTile + first) * p.d;
  uint16_t* out = is_v ? p.dv + hk * p.dv_head : p.dk + hk * p.dk_head;
  const int64_t tok = is_v ? p.dv_tok : p.dk_tok;
  for (int i = (int)threadIdx.x; i < rows * parts; i += 256) {
    const float4* src = reinterpret_cast<const float4*>(base + 8 * (size_t)i);   // (rows are p.d = 8 parts floats apart)
    float4 a = src[0], c = src[1];
#pragma unroll 4
    for (int k = 1; k < n; ++k) {
      const float4* y = reinterpret_cast<const float4*>(base + k * step + 8 * (size_t)i);
      const float4 ya = y[0], yc = y[1];
      a = make_float4(a.x + ya.x, a.y + ya.y, a.z + ya.z, a.w + ya.w);
      c = make_float4(c.x + yc.x, c.y + yc.y, c.z + yc.z, c.w + yc.w);
    }
    put(out + ((int64_t)it.start + kTile * it.c + first + i / parts) * tok + 8 * (i % parts), a, c, is_v ? 1.f : p.scale);
  }
}

template <int D, bool F16, int SLOTS, int SCORE>
cudaError_t launch_packed_bwd_d(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                const CUtensorMap& tdo, const CUtensorMap& tdq,
                                const PackedBwdParams& p, cudaStream_t s) {
  using L = PackedBwdLayout<D>;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static PerDeviceOnce smem_set;
  e = once_per_device(smem_set, dev, [] {
    return cudaFuncSetAttribute(fa_packed_bwd_kernel<D, F16, SLOTS, SCORE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                L::kSmemBytes);
  });
  if (e != cudaSuccess) return e;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  PackedBwdParams q = p;
  // Q and dO (16-bit) and the fp32 dQ accumulator of a key/value head's G query
  // heads are re-read by all of its key tiles
  q.group = l2_head_group(8.0 * p.total * p.d * p.G, p.Hk) * p.parts;
  const dim3 tiles((unsigned)p.cap_tiles * (unsigned)p.Hq);
  // Only the main kernel is launched ahead of its predecessor's end. With the two
  // passes launched ahead as well, their blocks are scheduled between those of a
  // kernel still running: forward and backward of 16 documents 308 us against
  // 286, of two long sequences 1273 against 1250 (one short one 25.5 against 25.8).
  // 16 lanes cover d <= 128, 8 cover d <= 64
  // (up to kDirect sequences the passes' blocks read the bounds themselves)
  const bool direct = p.B <= kDirect;
  if constexpr (SCORE != kScorePlain) e = launch_packed_dots<D, F16, SCORE>(tq, tk, tv, tdo, q, sms, s);
  else e = launch_pdl(false, direct ? packed_bwd_pre_kernel<D / 8, F16, SLOTS> : packed_bwd_pre_kernel<D / 8, F16, 0>, tiles,
                 dim3(256), 0, s, q);
  if (e != cudaSuccess) return e;
  // a CTA per item where items are taken by cancelling CTAs, else one per SM
  const long long most = (long long)p.cap_tiles * p.Hk * p.parts;
  e = launch_pdl(true, fa_packed_bwd_kernel<D, F16, SLOTS, SCORE>, dim3((unsigned)(direct || most < sms ? most : sms)),
                 dim3(kBwdThreads), L::kSmemBytes, s, tq, tk, tv, tdo, tdq, q);
  if (e != cudaSuccess) return e;
  if (p.parts == 1)
    return launch_pdl(false, direct ? packed_bwd_dq_kernel<F16, false, SLOTS, false> : packed_bwd_dq_kernel<F16, false, 0, false>,
                      tiles, dim3(256), 0, s, q);
  const unsigned sums = (unsigned)p.cap_tiles * (unsigned)p.Hk * 2u * (kTile / kSumRows);
  return launch_pdl(false, packed_bwd_dq_kernel<F16, true, SLOTS, SCORE != kScorePlain>, dim3(tiles.x + sums), dim3(256), 0, s, q);
}

template <int SCORE>
cudaError_t launch_packed_bwd_score(bool f16, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                    const CUtensorMap& tdo, const CUtensorMap& tdq, const PackedBwdParams& p,
                                    cudaStream_t s) {
  auto run = [&](auto many) -> cudaError_t {
    constexpr int SLOTS = many ? kManySlots : 1;
    if (p.d <= 64)
      return f16 ? launch_packed_bwd_d<64, true, SLOTS, SCORE>(tq, tk, tv, tdo, tdq, p, s)
                 : launch_packed_bwd_d<64, false, SLOTS, SCORE>(tq, tk, tv, tdo, tdq, p, s);
    return f16 ? launch_packed_bwd_d<128, true, SLOTS, SCORE>(tq, tk, tv, tdo, tdq, p, s)
               : launch_packed_bwd_d<128, false, SLOTS, SCORE>(tq, tk, tv, tdo, tdq, p, s);
  };
  if (SCORE != kScorePlain || packed_many(p.B)) return run(std::true_type{});
  if constexpr (SCORE == kScorePlain) return run(std::false_type{});
  return cudaErrorInvalidValue;
}

}  // namespace

}  // namespace fa
