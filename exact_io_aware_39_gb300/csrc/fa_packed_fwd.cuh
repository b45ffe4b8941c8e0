// Forward pass over packed sequences with grouped heads, for sm_103a
// (tcgen05 tensor cores, TMEM accumulators, TMA staging).
//
// The arithmetic of a 128-row query tile is that of fa_fwd.cu: S = Q K_j^T in
// TMEM, one softmax warpgroup per query tile (thread = row) that writes P packed
// to 16 bits into TMEM, O += P V_j in TMEM, the reference maximum moved only
// past 2^8. What is different:
//   * a work item is two query tiles that share their K and V loads: the same
//     tile of two neighbouring query heads of one key/value head where the group
//     size is even (both then end at the same key tile, and a sequence of one
//     tile still fills both softmax groups), else two neighbouring tiles of a
//     head. Calls of few query tiles take one to an item instead and share its key
//     tiles out between the groups, whose sums are joined from TMEM (SPLIT);
//   * the items of a call are listed on the device (the lengths are there),
//     heaviest first (but for prefixes, which the order does not know): for up to 128 sequences by every producer warp for itself
//     (DirectList), for more by a plan kernel. A CTA takes its own item, then,
//     as it gets ready for one, the next of a counter that the plan kernel zeroed
//     or, without one, a CTA of the grid that has not started, cancelled through
//     cluster launch control (dealing the sorted list out in a fixed snake was
//     12 % slower on one sequence of 16384 tokens, 32 heads, d = 128);
//   * no role waits for another at the end of an item. Items pass through a
//     ring, every barrier phase runs on across them, and a query tile's
//     Q buffer goes back to the producer behind its last S, so the next item's
//     loads and first S products run while this one's O is read out;
//   * O goes from registers to global memory, four lanes writing 64 bytes of a
//     row (a transpose across the lane quad), which needs no staging buffer and
//     ends at a sequence's end without a second path;
//   * tensors are [token, head, d] with any strides: a tile is a 3-D TMA box of
//     one head and 128 tokens. It may run into the next sequence: keys past the
//     end are masked in S, and their rows of V are zeroed in shared memory before
//     the product (a zero weight times a NaN that lies there would be NaN).
//
// Bound: 4 d operations per visible pair on the tensor cores, and one
// exponential per pair, which at d = 64 takes as long (16 per clock and SM); for
// short sequences an item's way from its loads to its O. Measured (the kernel,
// replayed a few times from a graph), bf16, causal, 32 query and 8 key/value heads,
// d = 128: one sequence of 16384 tokens 1.22 ms (1.81 PFLOP/s, 95 % of the measured
// dense peak; call after call for seconds, under the power cap, 1.34 ms); 24 sequences
// of 16-2048 tokens 106 us (1.07 PFLOP/s). The second was 150 + 10 us with a barrier of all roles
// around each item and the plan kernel for every call, 124 with the ring and the
// pairs of heads (144 with pairs of tiles), and the rest is code size: an item
// passes through all of the kernel's code, which at 96 KB missed the instruction
// cache all the way and now has 55.
#pragma once

#include "fa_packed.cuh"
#include "fa_packed_rows.cuh"

#include <type_traits>

namespace fa {

namespace {

constexpr float kRescaleThreshold = 8.0f; // log2 units
constexpr float kSpecSumLimit = 256.0f;    // 2^kRescaleThreshold

template <int D, bool SPLIT, bool PRE>
struct PackedFwdLayout {
  // Softmax warpgroups of a query tile: one, or for scores of their own two with
  // half of a row's columns each
  static constexpr int kParts = PRE ? 2 : 1;
  static constexpr int kOther = 8 * kParts;                     // the first of the four warps behind them
  static constexpr int kThreads = 32 * (kOther + 4);
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kHalves = D / 64;
  // separate K and V rings; the K ring is the deeper one, since the S MMAs
  // that read K come first
  static constexpr int kStagesK = (D == 64) ? 5 : 3;
  static constexpr int kStagesV = (D == 64) ? 4 : 2;
  // Q buffers of each query tile: at d = 64 two, at d = 128 the shared memory
  // holds one. At d = 64, S_0, S_1 (128 columns each) and O_0, O_1 (64 each)
  // leave 128 TMEM columns, which give each Q tile's P columns of their own:
  // S_t is then free as soon as its softmax group has read it into registers,
  // and the next S_t is computed while that group works on this one. At d = 128
  // the four regions fill TMEM and P is packed over S in place.
  // For scores of their own, whose softmax takes longer than the products, P has its
  // columns at d = 128 too: the two query tiles share one S region there, which is
  // free as soon as one tile's groups have read it into registers, so that the next
  // S is computed while they work.
  static constexpr bool kOwnP = (D == 64) || PRE;
  static constexpr bool kSharedS = PRE && D == 128;
  static constexpr int kQBuf = (D == 64) ? 2 : 1;
  static constexpr int kItemRing = 4;
  static constexpr int kQ = 0;                              // [2][kQBuf] tiles
  static constexpr int kK = kQ + 2 * kQBuf * kTileBytes;
  static constexpr int kV = kK + kStagesK * kTileBytes;
  static constexpr int kBar = kV + kStagesV * kTileBytes;   // 8-byte mbarriers
  // barrier slots
  static constexpr int bQFull = 0;                    // [2][kQBuf]
  static constexpr int bQEmpty = bQFull + 2 * kQBuf;  // [2][kQBuf]: the tile's last S is complete
  static constexpr int bKFull = bQEmpty + 2 * kQBuf;
  static constexpr int bKEmpty = bKFull + kStagesK;
  static constexpr int bVFull = bKEmpty + kStagesK;
  static constexpr int bVEmpty = bVFull + kStagesV;
  static constexpr int bSFull = bVEmpty + kStagesV;   // [2]
  static constexpr int bPFull = bSFull + 2;           // [2], 4 arrivals (warps)
  static constexpr int bOFinal = bPFull + 2;          // [2]
  static constexpr int bSFree = bOFinal + 2;          // [2], 4: S_t read into registers (own P columns only)
  static constexpr int bPVDone = bSFree + 2;          // [2] O_t += P_t V complete (own P columns only)
  static constexpr int bPHalf = bPVDone + 2;          // [2], 4: P_t of the first 64 keys is in TMEM (P over S only)
  static constexpr int bItemFull = bPHalf + 2;        // [kItemRing]
  static constexpr int bItemEmpty = bItemFull + kItemRing;   // [kItemRing], 10: V producer, MMA and softmax warps
  static constexpr int bClc = bItemEmpty + kItemRing;        // the next item's cancellation answer has arrived
  // split keys: O_1 and the second group's statistics are complete; they have been read
  static constexpr int bStats = bClc + 1;             // 4 arrivals
  static constexpr int bJoined = bStats + 1;          // 4
  static constexpr int bDrain = SPLIT ? bJoined + 1 : bStats;
  static constexpr int kNumBars = bDrain + 1;
  static constexpr int kMisc = (kBar + 8 * kNumBars + 15) & ~15;   // tmem slot, abort flag, -, wait limit
  static constexpr int kRing = kMisc + 16;            // [kItemRing] x {first row, length, unit or -1, head}
  static constexpr int kClc = kRing + 16 * kItemRing;   // 16-byte answer of a launch cancellation
  static constexpr int kStats = kClc + 16;              // [128] (reference, sum) of the second group's rows
  // PRE: what a tile's two groups tell each other, [query tile] [half] [128], and,
  // split, the second tile's references [128]
  static constexpr int kEx = kClc + 16, kExRef = kEx + 4 * kTile * 4;
  static constexpr int kSmemBytes = PRE ? kExRef + (SPLIT ? 4 * kTile : 0) : kStats + (SPLIT ? 8 * kTile : 0);
  static_assert(kSmemBytes <= 232448, "shared memory budget");
};

template <int D, bool F16, int SLOTS, bool SPLIT, int SCORE>
__global__ void __launch_bounds__(PackedFwdLayout<D, SPLIT, SCORE != kScorePlain>::kThreads, 1)
fa_packed_fwd_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                     const __grid_constant__ CUtensorMap tv, const PackedFwdParams p) {
  using L = PackedFwdLayout<D, SPLIT, SCORE != kScorePlain>;
  // With P over S (d = 128), P of a tile's first 64 keys goes to the tensor
  // core before the rest is formed, and its half of P V runs meanwhile; the
  // softmax then always takes the row max first, since P may not be formed
  // again once half of it has been used
  // (scores of their own have a warpgroup for either half, which hand P over together)
  constexpr bool PRE = SCORE != kScorePlain;
  constexpr bool kHalfP = !L::kOwnP && !PRE;
  constexpr int kOtherRegs = PRE ? kHalfOtherRegs : kRowOtherRegs;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);

  const int tid = threadIdx.x;
  // (from a shuffle, so that the compiler knows it to be the same in all lanes:
  // the operands of an MMA are uniform registers, and in a branch that it takes
  // for divergent each MMA costs some 40 instructions more)
  const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  const int lane = tid & 31;

  auto bar = [&](int i) -> uint32_t { return sbase + L::kBar + 8u * (uint32_t)i; };
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  volatile uint32_t* abort_flag = misc + 1;
  volatile int* ring = reinterpret_cast<volatile int*>(smem + L::kRing);
  Ctl ctl{p.err, abort_flag};

  if ((sbase & 1023u) != 0u) {   // uniform across the CTA: nothing has started yet
    if (tid == 0) {
      uint32_t dummy = 0;   // report_error writes only the abort flag
      Ctl c0{p.err, &dummy};
      report_error(c0, kErrSmemAlign, 310);
    }
    return;
  }

  if (tid == 0) {
    auto arrivals = [](int i) -> uint32_t {
      if ((i >= L::bPFull && i < L::bPFull + 2) || (i >= L::bSFree && i < L::bSFree + 2) ||
          (i >= L::bPHalf && i < L::bPHalf + 2) || (SPLIT && (i == L::bStats || i == L::bJoined)))
        return 4u * L::kParts;
      return i >= L::bItemEmpty && i < L::bItemEmpty + L::kItemRing ? 2u + 8u * L::kParts : 1u;
    };
    for (int i = 0; i < L::kNumBars; ++i) mbar_init(bar(i), arrivals(i));
    abort_flag[0] = 0u;
    abort_flag[2] = p.wait_us;   // the wait limit, read by the slow path of every wait
    fence_mbar_init();
  }
  if (warp == L::kOther + 1) {
    tmem_alloc(smem_u32(misc), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();   // the barriers are initialised and TMEM allocated
  tc_fence_after();
  const uint32_t tmem = misc[0];
  // global memory is read and written only from here on: what the previous
  // kernel in the stream wrote is complete and visible
  grid_dep_wait();
  grid_dep_launch();

  // Item k of this CTA from the ring; w.c < 0 when none is left or a wait
  // failed (then ok is false too). Executed by whole warps.
  auto take_item = [&](int k, Pair<SPLIT, PRE>& w) -> bool {
    const int rs = k % L::kItemRing;
    w.c = -1;
    if (!bar_wait_warp(bar(L::bItemFull + rs), (uint32_t)(k / L::kItemRing) & 1u, ctl, 319)) return false;
    w.start = __shfl_sync(0xFFFFFFFFu, ring[4 * rs], 0);   // (the same in all lanes, as the compiler then knows)
    w.len = __shfl_sync(0xFFFFFFFFu, ring[4 * rs + 1], 0);
    w.c = __shfl_sync(0xFFFFFFFFu, ring[4 * rs + 2], 0);
    w.head = __shfl_sync(0xFFFFFFFFu, ring[4 * rs + 3], 0);
    w.finish(p.pair_heads != 0, p.causal != 0, PRE && p.score.slopes != nullptr);
    mbar_arrive_warp(bar(L::bItemEmpty + rs));
    return true;
  };

  if (warp == L::kOther) {
    // ------------------------------------------------------------ items, Q and K producer
    regs_dec<kOtherRegs>();
    if (lane == 0) {
      tma_prefetch_map(&tq);
      tma_prefetch_map(&tk);
    }
    // The work order walks groups of p.group heads whose K and V fit in L2
    // together, within a group the list heaviest first, and for each unit the
    // heads of the group.
    const bool direct = p.B <= kDirect;
    DirectList<SLOTS, PRE> dl;
    int n_items = 0;
    if (direct) {
      dl.init(p.cu, p.score.prefix, p.B, p.total, SPLIT || p.pair_heads ? kTile : 2 * kTile, p.cap_items, p.causal != 0, p.err);
      n_items = dl.items;
    } else {
      n_items = p.plan->items;
    }
    const int total = n_items * p.heads;
    int nk = 0;                  // K loads issued
    int nq0 = 0, nq1 = 0;        // Q loads issued per query tile
    bool clc_out = false;        // a cancellation answer is outstanding
    uint32_t clc = 0u;           // answers received
    bool ok = true;
    for (int k = 0; ok; ++k) {
      const int rs = k % L::kItemRing;
      if (k >= L::kItemRing &&
          !(ok = bar_wait_warp(bar(L::bItemEmpty + rs), (uint32_t)(k / L::kItemRing - 1) & 1u, ctl, 313)))
        break;
      int item = (int)blockIdx.x;
      if (k > 0 && !direct) {
        item = (int)gridDim.x + __shfl_sync(0xFFFFFFFFu, lane == 0 ? (int)atomicAdd(&p.plan->sched, 1u) : 0, 0);
      } else if (k > 0) {
        // (the grid is sized for the most items these bounds can have: CTAs past
        // the list are cancelled too, until none is left)
        do {
          if (lane == 0) {
            mbar_arrive_expect_tx(bar(L::bClc), 16u);
            clc_try_cancel(sbase + L::kClc, bar(L::bClc));
          }
          __syncwarp();
          clc_out = true;
          if (!(ok = bar_wait_warp(bar(L::bClc), clc & 1u, ctl, 309))) break;
          clc_out = false;
          ++clc;
          item = __shfl_sync(0xFFFFFFFFu, clc_first_ctaid_x(sbase + L::kClc), 0);
        } while (item >= total);
        if (!ok) break;
        if (item < 0) item = total;
      }
      Pair<SPLIT, PRE> w;
      w.c = -1;
      int ring_c = -1;
      if (item < total) {
        int head = 0;
        const int idx = split_grouped(item, p.group, n_items, p.heads, &head);
        const PackedItem pi = direct ? dl.at(idx, p.causal != 0) : p.items[idx];
        w.start = pi.start;
        w.len = pi.len;
        w.c = pi.c;
        if (PRE && direct) w.c = with_prefix(pi.c, dl.prefix);
        ring_c = w.c;
        w.head = head;
        w.finish(p.pair_heads != 0, p.causal != 0, PRE && p.score.slopes != nullptr);
      }
      if (lane == 0) {
        ring[4 * rs] = w.start;
        ring[4 * rs + 1] = w.len;
        ring[4 * rs + 2] = ring_c;
        ring[4 * rs + 3] = w.head;
        mbar_arrive(bar(L::bItemFull + rs));   // (release: the ring entry is visible to the waiters)
      }
      if (w.c < 0) break;
      const int hk = w.hq(0) / p.G;
      // Q can only be loaded behind the last S of the item before: it is
      // brought into L2 until then
      if (k >= L::kQBuf)
#pragma unroll 1
        for (int t = 0; t < 2; ++t)
          for (int a = 0; w.has(t) && a < L::kHalves; ++a)
            tma_prefetch_3d_w(&tq, 64 * a, w.hq(t), w.start + kTile * w.qi(t));
#pragma unroll 1
      for (int e = 0; e < w.n && ok; ++e) {
        if (p.stall != 0u && e >= 1) { ok = false; break; }   // test of the timeout path: K of entry 1 never comes
        // K of key tile e, once the MMAs of the entry that used the slot
        // before (of this item or an earlier one) have read it
        const int sk = nk % L::kStagesK;
        if (nk >= L::kStagesK &&
            !(ok = bar_wait_warp(bar(L::bKEmpty + sk), (uint32_t)(nk / L::kStagesK - 1) & 1u, ctl, 311)))
          break;
        mbar_arrive_expect_tx_w(bar(L::bKFull + sk), L::kTileBytes);
        for (int a = 0; a < L::kHalves; ++a)
          tma_load_3d_w(sbase + L::kK + sk * L::kTileBytes + a * 16384, &tk, bar(L::bKFull + sk), 64 * a, hk,
                        w.start + kTile * w.tile(e));
        ++nk;
        // the item's Q tiles behind its first K, which seldom waits; a tile's
        // buffer is free once the last S of the item before has read it
#pragma unroll 1
        for (int t = 0; e == 0 && t < 2 && ok; ++t) {
          if (!w.has(t)) continue;
          const int nt = t ? nq1 : nq0, slot = t * L::kQBuf + nt % L::kQBuf;
          if (nt >= L::kQBuf &&
              !(ok = bar_wait_warp(bar(L::bQEmpty + slot), (uint32_t)(nt / L::kQBuf - 1) & 1u, ctl, 310)))
            break;
          mbar_arrive_expect_tx_w(bar(L::bQFull + slot), L::kTileBytes);
          for (int a = 0; a < L::kHalves; ++a)
            tma_load_3d_w(sbase + L::kQ + slot * L::kTileBytes + a * 16384, &tq, bar(L::bQFull + slot), 64 * a, w.hq(t),
                          w.start + kTile * w.qi(t));
          (t ? nq1 : nq0) += 1;
        }
      }
    }
    // every load and cancellation request issued has completed before the CTA
    // exits; loads were issued in ring order, so the last load into slot s was
    // number s + S * floor((n - 1 - s) / S)
    if (lane == 0) {
      if (clc_out) drain_wait(bar(L::bClc), clc & 1u);
#pragma unroll 1
      for (int i = 0; i < 2 * L::kQBuf; ++i) {
        const int nt = i < L::kQBuf ? nq0 : nq1, b = i % L::kQBuf;
        if (b < nt) drain_wait(bar(L::bQFull + i), (uint32_t)((nt - 1 - b) / L::kQBuf) & 1u);
      }
#pragma unroll 1
      for (int s = 0; s < L::kStagesK && s < nk; ++s)
        drain_wait(bar(L::bKFull + s), (uint32_t)((nk - 1 - s) / L::kStagesK) & 1u);
    }
  } else if (warp == L::kOther + 2) {
    // ------------------------------------------------------------ V producer
    // (its own warp, so that the K ring can run ahead of the V ring)
    regs_dec<kOtherRegs>();
    if (lane == 0) tma_prefetch_map(&tv);
    int nv = 0;
    Pair<SPLIT, PRE> w;
    bool ok = true;
    for (int k = 0; ok && take_item(k, w) && w.c >= 0; ++k) {
      const int hk = w.hq(0) / p.G;
#pragma unroll 1
      for (int e = 0; e < w.n; ++e) {
        const int sv = nv % L::kStagesV;
        if (nv >= L::kStagesV &&
            !(ok = bar_wait_warp(bar(L::bVEmpty + sv), (uint32_t)(nv / L::kStagesV - 1) & 1u, ctl, 312)))
          break;
        mbar_arrive_expect_tx_w(bar(L::bVFull + sv), L::kTileBytes);
        for (int a = 0; a < L::kHalves; ++a)
          tma_load_3d_w(sbase + L::kV + sv * L::kTileBytes + a * 16384, &tv, bar(L::bVFull + sv), 64 * a, hk,
                        w.start + kTile * w.tile(e));
        ++nv;
      }
    }
    if (lane == 0)
#pragma unroll 1
      for (int s = 0; s < L::kStagesV && s < nv; ++s)
        drain_wait(bar(L::bVFull + s), (uint32_t)((nv - 1 - s) / L::kStagesV) & 1u);
  } else if (warp == L::kOther + 1) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp runs the schedule; one elected lane issues each MMA and
    // commit. At entry e, for each Q tile t, first the pending O_t += P_t V of
    // t's previous entry (waiting for P_t), then S_t = Q_t K_e^T. For dense rows
    // this is
    //   PV0(e-1), S0(e), PV1(e-1), S1(e), PV0(e), ...
    // so that while one softmax group works the tensor core runs the other
    // tile's products; with P columns of their own both S of an entry come
    // before both PV, so S_t(e+1) is computed while group t still works on
    // S_t(e). The last PVs of an item stay pending into the next one, unless
    // its first loads are not there yet.
    regs_dec<kOtherRegs>();
    constexpr uint32_t idS = idesc_16<F16>(128, 128, false, false);
    constexpr uint32_t idO = idesc_16<F16>(128, D, false, true);
    const uint32_t tS[2] = {tmem + 0u, tmem + (L::kSharedS ? 0u : 128u)};
    const uint32_t tO[2] = {tmem + 256u, tmem + 256u + (uint32_t)D};
    // P_t: over S_t, or in columns of its own (after O_1; where S is shared, behind it)
    constexpr uint32_t kP0 = L::kSharedS ? 128u : 256u + 2u * D;
    const uint32_t tP[2] = {L::kOwnP ? tmem + kP0 : tS[0], L::kOwnP ? tmem + kP0 + 64u : tS[1]};
    const uint32_t dQ0 = desc_lo(desc_kmajor(sbase + L::kQ, 0));
    const uint32_t dK0 = desc_lo(desc_kmajor(sbase + L::kK, 0));
    const uint32_t dV0 = desc_lo(desc_mnmajor(sbase + L::kV, 0));
    constexpr uint32_t kSlotStep = (uint32_t)(L::kTileBytes >> 4);
    int nk = 0, nv = 0;              // K and V ring entries of the entries before this one
    int nq[2] = {0, 0};              // items with query tile t so far
    [[maybe_unused]] int last_s = -1;   // shared S: the tile of the last one
    uint32_t ns[2] = {0u, 0u}, npv[2] = {0u, 0u};   // S and PV groups issued per Q tile
    // the pending PV of each Q tile: its V ring entry or -1, whether it is the
    // item's first (overwrites O_t) and last, and the valid rows of a V tile
    // that the sequence ends in (else 0)
    int pend[2] = {-1, -1};
    bool pfirst[2] = {false, false}, plast[2] = {false, false};
    int ptail[2] = {0, 0};
    int zeroed = -1;                 // last V ring entry whose rows past the sequence were zeroed
    bool open = false;               // V ring entry nv - 1 has not gone back to the producer
    bool ok = true, more = true;
    Pair<SPLIT, PRE> w;
    for (int k = 0; ok && more; ++k) {
      if (!(ok = take_item(k, w))) break;
      more = w.c >= 0;
      const int n = more ? w.n : 0;
      const int tail = w.tail();
      const int tail_e = w.tile(w.nT - 1);   // the entry of the sequence's last key tile (tile() is its own inverse)
      const int last[2] = {w.last(0), w.has(1) ? w.last(1) : -1};   // t is live at entries 0 .. last
      // Q_t of this item: its buffer and phase
      auto q_slot = [&](int t) -> int { return t * L::kQBuf + nq[t] % L::kQBuf; };
      auto q_phase = [&](int t) -> uint32_t { return (uint32_t)(nq[t] / L::kQBuf) & 1u; };
      // Where this item's first loads are not there yet, its pending PVs go
      // before its first S, as an entry -1 without an S of its own. (The loop
      // holds each product's code once per query tile: an item passes through
      // every line of the kernel, and a larger one misses the instruction cache;
      // with copies of its own for the end of an item, items of one key tile
      // took 4.9 us instead of 4.2.)
      bool first = !more || SPLIT;   // (SPLIT: a pending product may belong to a group that this item does not have)
      if (!SPLIT && more) {
        const bool there = mbar_test(bar(L::bQFull + q_slot(0)), q_phase(0)) &&
                           mbar_test(bar(L::bKFull + nk % L::kStagesK), (uint32_t)(nk / L::kStagesK) & 1u);
        first = !__all_sync(0xFFFFFFFFu, there);
      }
      // entry e, for both query tiles (which = 2) or, SPLIT, for one group; a
      // constant, so that the products' operands stay uniform registers
      auto entry = [&](const int e, auto which) {
        constexpr int kWhich = which;
        const int sk = nk % L::kStagesK;
        bool k_ready = false;
        // S_t = Q_t K_e^T
        auto issue_s = [&](int t) -> bool {
          if constexpr (L::kSharedS) {
            if (last_s >= 0 && !bar_wait_warp(bar(L::bSFree + last_s), ((last_s ? ns[1] : ns[0]) - 1u) & 1u, ctl, 318)) return false;
            last_s = t;
          } else if (L::kOwnP && ns[t] > 0 && !bar_wait_warp(bar(L::bSFree + t), (ns[t] - 1u) & 1u, ctl, 318)) {
            return false;
          }
          if (e == w.first(t) && !bar_wait_warp(bar(L::bQFull + q_slot(t)), q_phase(t), ctl, 314)) return false;
          if (!k_ready && !bar_wait_warp(bar(L::bKFull + sk), (uint32_t)(nk / L::kStagesK) & 1u, ctl, 317)) return false;
          k_ready = true;
          tc_fence_after();
          const uint32_t dQ = dQ0 + (uint32_t)q_slot(t) * kSlotStep, dK = dK0 + (uint32_t)sk * kSlotStep;
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            mma_ss_lo(tS[t], dQ + (uint32_t)kmajor_step(ks), dK + (uint32_t)kmajor_step(ks), idS, ks > 0 ? 1u : 0u);
          mma_commit_w(bar(L::bSFull + t));
          if (e == last[t]) mma_commit_w(bar(L::bQEmpty + q_slot(t)));   // Q_t is no longer needed
          ++ns[t];
          return true;
        };
        // O_t += P_t V of the pending entry
        auto issue_pv = [&](int t) -> bool {
          const int v = pend[t], sv = v % L::kStagesV;
          pend[t] = -1;
          if (!bar_wait_warp(bar((kHalfP ? L::bPHalf : L::bPFull) + t), npv[t] & 1u, ctl, 315)) return false;
          if (!bar_wait_warp(bar(L::bVFull + sv), (uint32_t)(v / L::kStagesV) & 1u, ctl, 316)) return false;
          if (ptail[t] != 0 && zeroed != v) {
            zero_tail_rows<D>(smem + L::kV + sv * L::kTileBytes, ptail[t]);
            zeroed = v;
          }
          tc_fence_after();
          const uint32_t dV = dV0 + (uint32_t)sv * kSlotStep;
          const uint32_t acc0 = pfirst[t] ? 0u : 1u;
#pragma unroll
          for (int ks = 0; ks < kTile / 16; ++ks) {
            if (kHalfP && ks == kTile / 32) {   // the second half of P
              if (!bar_wait_warp(bar(L::bPFull + t), npv[t] & 1u, ctl, 315)) return false;
              tc_fence_after();
            }
            mma_ts_lo(tO[t], tP[t] + (uint32_t)ks * 8u, dV + (uint32_t)mnmajor_step(ks), idO, ks > 0 ? 1u : acc0);
          }
          if constexpr (L::kOwnP) mma_commit_w(bar(L::bPVDone + t));   // P_t may be rewritten, O_t rescaled
          if (plast[t]) mma_commit_w(bar(L::bOFinal + t));             // O_t is complete
          if constexpr (SPLIT) mma_commit_w(bar(L::bVEmpty + sv));     // V of the entry is this group's alone
          ++npv[t];
          return true;
        };
        // the entry's PV becomes the pending one once the one before it is on its way
        auto set_pending = [&](int t) {
          pend[t] = nv;
          pfirst[t] = e == w.first(t);
          plast[t] = e == last[t];
          ptail[t] = e == tail_e ? tail : 0;
        };
        auto on = [](int t) -> bool { return kWhich == 2 || t == kWhich; };
        if constexpr (L::kSharedS) {
          // S_0(e), PV_0(e - 1), S_1(e), PV_1(e - 1): S_1 waits until S_0 has been read,
          // which is after P_0(e - 1) was written. (A group reads its first S of an item
          // once its last O of the item before is written: there PV goes first.)
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (!on(t)) continue;
            if (ok && e <= 0 && pend[t] >= 0) ok = issue_pv(t);
            if (ok && e >= 0 && e <= last[t]) ok = issue_s(t);
            if (ok && e >= 0 && (t == 1 || kWhich == 0)) mma_commit_w(bar(L::bKEmpty + sk));   // K_e is no longer needed
            if (ok && pend[t] >= 0) ok = issue_pv(t);
            if (e >= 0 && e <= last[t]) set_pending(t);
          }
        } else if constexpr (L::kOwnP) {
#pragma unroll
          for (int t = 0; t < 2; ++t)
            if (ok && e >= 0 && e <= last[t] && on(t)) ok = issue_s(t);
          if (!ok) return;
          if (e >= 0) mma_commit_w(bar(L::bKEmpty + sk));   // K_e is no longer needed
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (ok && pend[t] >= 0 && on(t)) ok = issue_pv(t);
            if (e >= 0 && e <= last[t] && on(t)) set_pending(t);
          }
        } else {
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (ok && pend[t] >= 0 && on(t)) ok = issue_pv(t);
            if (ok && e >= 0 && e <= last[t] && on(t) && (ok = issue_s(t))) set_pending(t);
          }
          if (ok && e >= 0) mma_commit_w(bar(L::bKEmpty + sk));   // K_e is no longer needed
        }
        if (!ok) return;
        if (!SPLIT && open) mma_commit_w(bar(L::bVEmpty + (nv - 1) % L::kStagesV));   // both PVs of the entry before are issued
        open = e >= 0;
        if (e >= 0) {
          ++nk;
          ++nv;
        }
      };
      using Both = std::integral_constant<int, 2>;
      if constexpr (SPLIT) {
        entry(-1, Both{});
#pragma unroll 1
        for (int e = 0; e < n && ok; e += 2) {
          entry(e, std::integral_constant<int, 0>{});
          if (e + 1 < n && ok) entry(e + 1, std::integral_constant<int, 1>{});
        }
      } else {
#pragma unroll 1
        for (int e = first ? -1 : 0; e < n && ok; ++e) entry(e, Both{});
      }
      if (more) {
        ++nq[0];
        nq[1] += w.has(1) ? 1 : 0;
      }
    }
    // every MMA issued has completed before TMEM is freed
    mma_commit_w(bar(L::bDrain));
    drain_wait(bar(L::bDrain), 0);
  } else if (PRE && warp < L::kOther) {
    // ------------------------------------------------------------ softmax groups, scores of their own
    // Thread = row and half of its columns; the two groups of a query tile share a
    // row's reference (they agree on it for every tile) and add their sums at the end. After
    // each wait that one of them may fail they agree with group_all, so that they
    // always take the same branch and none waits where the other has left.
    if constexpr (PRE) {
    regs_inc<kHalfRegs>();
    const int t = warp >> 3, h = (warp >> 2) & 1;
    const int r = tid & 127;
    const uint32_t pair_bar = 1u + (uint32_t)t;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + (uint32_t)((L::kSharedS ? 0 : t * 128) + 64 * h) + lane_off;
    const uint32_t tO = tmem + 256u + (uint32_t)(t * D) + lane_off;
    const uint32_t tP = tmem + (L::kSharedS ? 128u : 256u + 2u * D) + 64u * (uint32_t)t + lane_off + 32u * (uint32_t)h;
    constexpr int kCols0 = D / 64;           // 32-column steps of O that a half rescales and writes
    const float sl2 = p.scale_log2;
    constexpr bool kNoBias = SCORE == kScoreCapOnly;
    constexpr float kFar = 4.f;
    // A move stops all rows of a query tile, so without a bias, in bf16, a reference starts up to
    // 16 above the largest score of an item's first tile: one that moves it has to pass that by 30.
    // (24 prompts of 16-2048 tokens, 32 / 8 heads, d = 128, a cap of 50, scores of a standard
    // deviation of 10: 191 us, 243 with a reference that starts at the largest and moves past 20.)
    const float head = kNoBias && !F16 ? p.score.head : 0.f;
    volatile float* ex = reinterpret_cast<volatile float*>(smem + L::kEx) + r;   // [query tile][half][128]
    uint32_t nS = 0u, nO = 0u;               // S tiles and final O read by this group
    uint32_t nJ = 0u;                        // SPLIT: items of two groups so far
    Pair<SPLIT, PRE> w;
    for (int k = 0;; ++k) {
      bool ok = take_item(k, w);
      ok = group_all(pair_bar, 256u, ok);
      if (!ok || w.c < 0) break;
      if (!w.has(t)) continue;
      const int qi = w.qi(t), last = w.last(t);
      const int row = kTile * qi + r;        // query index within the sequence
      const float slope2 = !kNoBias && p.score.slopes != nullptr ? p.score.slopes[w.hq(t)] * 1.4426950408889634f : 0.f;
      float m_ref = 0.f;
      float l = 0.f;
      for (int i = w.first(t); i <= last; i += SPLIT ? 2 : 1) {
        const bool begin = i == w.first(t);
        const int e = w.tile(i);
        ok = ok && bar_wait_warp(bar(L::bSFull + t), nS & 1u, ctl, 320 + t);
        tc_fence_after();
        uint32_t u[2][32];
        tmem_ld32(tS, u[0]);
        tmem_ld32(tS + 32u, u[1]);
        tmem_ld_wait(u[0]);
        tmem_ld_wait(u[1]);
        tc_fence_before();
        mbar_arrive_warp(bar(L::bSFree + t));   // this half of S_t is in registers
        // keys from column `lim` on are masked: they lie past the row and the
        // prefix (causal), or past the sequence (never all of a row's columns in a
        // tile; rows past the sequence are not stored)
        const bool partial = w.partial(e, qi);
        const int lim = (w.causal ? min(max(row + 1, w.pre), w.len) : w.len) - kTile * e - 64 * h;
        float2 sum4[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        uint32_t pk[2][16];
        // 2^x of 32 arguments; P goes to 16 bits (half a step per weight), the row sum
        // takes the unrounded values
        auto weights = [&](int hh) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float p0 = ex2(__uint_as_float(u[hh][2 * i]));
            const float p1 = ex2(__uint_as_float(u[hh][2 * i + 1]));
            sum4[i & 3] = __fadd2_rn(sum4[i & 3], make_float2(p0, p1));
            pk[hh][i] = pack2<F16>(p0, p1);
          }
        };
        // Capped scores without a bias: where no row can pass its reference by the threshold,
        // none moves, and no maximum of the capped scores is formed. The raw ones' bounds
        // them: their magnitude, which the choice of the tanh needs anyway, where the polynomial
        // holds (|tanh x| <= |x|), else their maximum.
        bool stays = false;
        if constexpr (kNoBias) {
          if (!begin) {
            float most;
            const bool small = cap_vote(u, p.score, partial, lim, row < w.len, most);
            if (small) most *= p.score.a0;
            else most = p.score.c2 * tanh_exp(row_max(u), p.score);
            stays = group_all(pair_bar, 256u, ok && (row >= w.len || most <= m_ref + kRefMove));
            if (stays && small && !partial) {
              // (in one piece, so that the polynomial of some scores runs beside the
              // exponentials of others)
#pragma unroll
              for (int hh = 0; hh < 2; ++hh)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  const float2 x = pair_of(u[hh], 2 * i);
                  const float2 a = __ffma2_rn(x, cap_small_factor2(x, p.score), make_float2(-m_ref, -m_ref));
                  const float p0 = ex2(a.x);
                  const float p1 = ex2(a.y);
                  sum4[i & 3] = __fadd2_rn(sum4[i & 3], make_float2(p0, p1));
                  pk[hh][i] = pack2<F16>(p0, p1);
                }
            } else if (stays) {
#pragma unroll
              for (int hh = 0; hh < 2; ++hh) {
                cap_args(u[hh], p.score, partial, lim - 32 * hh, small, -m_ref);
                weights(hh);
              }
            }
          }
        }
        if (!stays) {
          const ScoreTile st = score_tile<SCORE>(p.score, slope2, kTile * e + 64 * h, row, e < qi ? -1 : e > qi ? 1 : 0,
                                                 e == qi && (!w.causal || w.pre > kTile * e), partial, lim, row < w.len);
          // The exponents against the row's reference as it is, which moves only where
          // one passes it by more than the threshold, and in an item's first tile. (Where
          // the tile's largest bias lies kFar above it, against that: from a reference
          // that is far below, they would be rounded in its units.)
          const float above = kNoBias ? -INFINITY : score_base(p.score, slope2, kTile * e, row, e < qi ? -1 : e > qi ? 1 : 0);
          const float base = begin ? (above > -INFINITY ? above : 0.f) : above > m_ref + kFar ? above : m_ref;
          const float mx = score_args<SCORE, true>(u, p.score, sl2, st, -base);
          if (begin || kNoBias || !group_all(pair_bar, 256u, ok && base <= m_ref && mx <= kRefMove)) {
            // (the first group has read O_1 and what goes with it of the item before)
            if (SPLIT && t == 1 && begin && nJ > 0u) ok = ok && bar_wait_warp(bar(L::bJoined), (nJ - 1u) & 1u, ctl, 328);
            // the previous O_t += P_t V has completed: O_t may be rescaled
            if (!begin) ok = ok && bar_wait_warp(bar(L::bPVDone + t), (nS - 1u) & 1u, ctl, 326 + t);
            ex[kTile * (2 * t + h)] = mx;
            if (!(ok = group_all(pair_bar, 256u, ok))) break;
            tc_fence_after();
            const float top = fmaxf(mx, ex[kTile * (2 * t + (h ^ 1))]);
            const float up = begin ? 0.f : base - m_ref;
            const bool move = begin || top + up > (up > 0.f ? 0.f : kRefMove);
            float alpha = 1.f, shift = up;
            if (move) {
              const float by = (top > -INFINITY ? top : 0.f) + head;   // (0: nothing to move to)
              alpha = begin ? 0.f : ex2(m_ref - (base + by));
              shift = -by;
              m_ref = base + by;
              l *= alpha;
            }
            // (warp-collective: a warp rescales when any of its rows needs it, 16 columns
            // at a time beside the scores)
            if (!begin && __any_sync(0xFFFFFFFFu, move)) {
#pragma unroll 1
              for (uint32_t cc = 0; cc < 2 * kCols0; ++cc) {
                uint32_t o[16];
                tmem_ld16(tO + 32u * kCols0 * h + 16u * cc, o);
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                tmem_st16(tO + 32u * kCols0 * h + 16u * cc, o);
              }
            }
#pragma unroll
            for (int hh = 0; hh < 2; ++hh)
#pragma unroll
              for (int i = 0; i < 32; i += 2) put_pair(u[hh], i, __fadd2_rn(pair_of(u[hh], i), make_float2(shift, shift)));
          }
          weights(0);
          weights(1);
        }
        const float2 s4 = __fadd2_rn(__fadd2_rn(sum4[0], sum4[1]), __fadd2_rn(sum4[2], sum4[3]));
        l += s4.x + s4.y;
        // P's columns are free once the product before has read them
        if (nS > 0u) ok = ok && bar_wait_warp(bar(L::bPVDone + t), (nS - 1u) & 1u, ctl, 326 + t);
        tc_fence_after();
        tmem_st16(tP, pk[0]);
        tmem_st16(tP + 16u, pk[1]);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive_warp(bar(L::bPFull + t));
        ++nS;
      }
      // O / l and the LSE, once the last PV has completed; a half writes half of the
      // columns
      if (ok) ok = bar_wait_warp(bar(L::bOFinal + t), nO & 1u, ctl, 324 + t);
      // (the other half has read what it needed: the last PV waited for its P)
      if (ok) ex[kTile * (2 * t + h)] = l;
      const bool join = SPLIT && w.has(1);
      float* ref1 = reinterpret_cast<float*>(smem + L::kExRef);
      if (SPLIT && join && t == 1 && h == 0 && ok) ref1[r] = m_ref;
      ok = group_all(pair_bar, 256u, ok);
      if (!ok) break;
      ++nO;
      tc_fence_after();
      float w0 = 1.f, w1 = 0.f;
      if (SPLIT && join && t == 1) {
        // (the sums stay where the first group finds them until it has joined them)
        tc_fence_before();
        mbar_arrive_warp(bar(L::bStats));
        ++nJ;
        continue;
      }
      l += ex[kTile * (2 * t + (h ^ 1))];
      if constexpr (SPLIT) {
        if (join) {
          ok = bar_wait_warp(bar(L::bOFinal + 1), nJ & 1u, ctl, 325) && bar_wait_warp(bar(L::bStats), nJ & 1u, ctl, 329);
          ok = group_all(pair_bar, 256u, ok);
          if (!ok) break;
          tc_fence_after();
          const float m1 = ref1[r], l1 = ex[kTile * 2] + ex[kTile * 3];
          ++nJ;
          const float M = fmaxf(m_ref, m1), ref = M == -INFINITY ? 0.f : M;
          w0 = ex2(m_ref - ref);
          w1 = ex2(m1 - ref);
          l = fmaf(w0, l, w1 * l1);
          m_ref = M;
        }
      }
      const float inv_l = 1.f / l;
      const int s4 = lane & 3;
      const int row0 = kTile * qi + 32 * (warp & 3) + (lane & ~3);   // the quad's first row
      uint16_t* op = p.o + (int64_t)(w.start + row0) * p.o_tok + w.hq(t) * p.o_head + 8 * s4;
#pragma unroll 1
      for (int cc = kCols0 * h; cc < kCols0 * (h + 1); ++cc) {
        uint32_t o[32];
        tmem_ld32(tO + 32u * cc, o);
        tmem_ld_wait(o);
        if constexpr (SPLIT) {
          if (join) {
            uint32_t o1[32];
            tmem_ld32(tO + (uint32_t)D + 32u * cc, o1);
            tmem_ld_wait(o1);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              o[i] = __float_as_uint(fmaf(w1, __uint_as_float(o1[i]), w0 * __uint_as_float(o[i])));
          }
        }
        uint32_t x[4][4];   // [word of a chunk][chunk of this row, then row of the quad]
#pragma unroll
        for (int wd = 0; wd < 4; ++wd) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            x[wd][j] = pack2<F16>(__uint_as_float(o[8 * j + 2 * wd]) * inv_l, __uint_as_float(o[8 * j + 2 * wd + 1]) * inv_l);
          quad_transpose(x[wd], (uint32_t)s4);
        }
        if (32 * cc + 8 * s4 < p.d) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (row0 + j < w.len)
              *reinterpret_cast<uint4*>(op + j * p.o_tok + 32 * cc) = make_uint4(x[0][j], x[1][j], x[2][j], x[3][j]);
        }
      }
      if (h == 0 && row < w.len)
        p.lse[(size_t)w.hq(t) * p.total + w.start + row] = (m_ref + log2f(l)) * 0.69314718055994531f;
      tc_fence_before();   // (the next PV of this tile waits for these groups' next P)
      if (join) mbar_arrive_warp(bar(L::bJoined));
    }
    }
  } else if (!PRE && warp < 8) {
    // ------------------------------------------------------------ softmax groups
    regs_inc<kSoftmaxRegs>();
    const int t = warp >> 2;                 // Q tile of this warpgroup
    const int r = tid & 127;                 // row within the tile = TMEM lane
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + (uint32_t)(t * 128) + lane_off;
    const uint32_t tO = tmem + 256u + (uint32_t)(t * D) + lane_off;
    const uint32_t tP = L::kOwnP ? tmem + 256u + 2u * D + 64u * (uint32_t)t + lane_off : tS;
    const float sl2 = p.scale_log2;
    uint32_t nS = 0u, nO = 0u;               // S tiles and final O read by this group
    uint32_t nJ = 0u;                        // SPLIT: items of two groups so far
    bool ok = true;
    Pair<SPLIT, PRE> w;
    for (int k = 0; ok && take_item(k, w) && w.c >= 0; ++k) {
      if (!w.has(t)) continue;
      const int qi = w.qi(t), last = w.last(t);
      const int row = kTile * qi + r;        // query index within the sequence
      float m_ref = -INFINITY;
      float l = 0.f;
      for (int e = w.first(t); e <= last; e += SPLIT ? 2 : 1) {
        const uint32_t n = (uint32_t)(e - w.first(t));   // 0: the first S tile of this item
        if (!(ok = bar_wait_warp(bar(L::bSFull + t), nS & 1u, ctl, 320 + t))) break;
        tc_fence_after();
        float x[128];
        {
          uint32_t u0[32], u1[32], u2[32], u3[32];
          tmem_ld32(tS + 0u, u0);
          tmem_ld32(tS + 32u, u1);
          tmem_ld32(tS + 64u, u2);
          tmem_ld32(tS + 96u, u3);
          tmem_ld_wait(u0);
          tmem_ld_wait(u1);
          tmem_ld_wait(u2);
          tmem_ld_wait(u3);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            x[i] = __uint_as_float(u0[i]);
            x[32 + i] = __uint_as_float(u1[i]);
            x[64 + i] = __uint_as_float(u2[i]);
            x[96 + i] = __uint_as_float(u3[i]);
          }
        }
        if constexpr (L::kOwnP) {   // S_t is in registers: the next S_t may be computed
          tc_fence_before();
          mbar_arrive_warp(bar(L::bSFree + t));
        }
        if (SPLIT && t == 1 && n == 0u && nJ > 0u) {
          // the first group has read O_1 of the item before: its product may be overwritten
          if (!(ok = bar_wait_warp(bar(L::bJoined), (nJ - 1u) & 1u, ctl, 328))) break;
          tc_fence_after();
        }
        if (w.partial(e, qi)) {
          // a key is masked when it lies past the row (causal) or past the
          // sequence: key >= min(row + 1, length), i.e. column i >= lim (never
          // all of a row's columns; rows past the sequence are not stored)
          const int lim = (w.causal ? min(row + 1, w.len) : w.len) - kTile * e;
#pragma unroll
          for (int i = 0; i < 128; ++i)
            if (i >= lim) x[i] = -INFINITY;
        }
        if (L::kOwnP && nS > 0) {
          // the previous O_t += P_t V has completed (of this item or the last
          // one): O_t may be rescaled and the P_t columns rewritten
          if (!bar_wait_warp(bar(L::bPVDone + t), (nS - 1u) & 1u, ctl, 326 + t)) { ok = false; break; }
          tc_fence_after();
        }
        // Two passes at most (at d = 64; at d = 128 only pass 1).
        // Pass 0 (not for a row block's first tile) takes the
        // exponentials with the current reference max: if every row of the warp
        // then sums to less than 2^8, no score exceeds the reference by the
        // rescale threshold, so the row max would not have moved it and P is
        // exactly what pass 1 would give. Otherwise pass 1 takes the row max,
        // moves the reference (rescaling O) where it grew past the threshold,
        // and redoes the exponentials (the whole warp: the TMEM stores are
        // warp-collective). This saves the row max on most tiles.
        float s_row = 0.f;
        // (when half of P goes ahead: always the row max)
#pragma unroll 1
        for (int pass = (n == 0 || kHalfP) ? 1 : 0; pass < 2; ++pass) {
          if (pass == 1) {
            // row max with three-input max: 8 independent chains over 128 scores
            float mx8[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) mx8[k] = x[k];
#pragma unroll
            for (int i = 8; i < 120; i += 16)
#pragma unroll
              for (int k = 0; k < 8; ++k) mx8[k] = fmax3(mx8[k], x[i + k], x[i + 8 + k]);
#pragma unroll
            for (int k = 0; k < 8; ++k) mx8[k] = fmaxf(mx8[k], x[120 + k]);
            const float mx = fmax3(fmax3(mx8[0], mx8[1], mx8[2]), fmax3(mx8[3], mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7]));
            const float m_new = mx * sl2;
            // move the reference max only when the row max grew by more than the
            // threshold; the O rescale is warp-collective (tcgen05.ld/st), so a
            // warp rescales when any of its rows needs it (alpha = 1 for the rest)
            const bool move = (n == 0) || (m_new > m_ref + kRescaleThreshold);
            float alpha = 1.f;
            if (move) {
              alpha = (n == 0 || m_ref == -INFINITY) ? 0.f : ex2(m_ref - m_new);
              l *= alpha;
              m_ref = m_new;
            }
            if (n > 0 && __any_sync(0xFFFFFFFFu, move)) {
              uint32_t u[32];
#pragma unroll
              for (int cc = 0; cc < D / 32; ++cc) {
                tmem_ld32(tO + 32u * cc, u);
                tmem_ld_wait(u);
#pragma unroll
                for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(__uint_as_float(u[i]) * alpha);
                tmem_st32(tO + 32u * cc, u);
              }
              tmem_st_wait();
            }
          }
          const float ref = (m_ref == -INFINITY) ? 0.f : m_ref;
          // packed fp32 pairs (one f32x2 instruction per two keys) for the
          // exponent arguments and the row sum: the softmax is issue-bound
          const float2 sl2x2 = make_float2(sl2, sl2);
          const float2 nref2 = make_float2(-ref, -ref);
          float2 sum4[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            uint32_t pk[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float2 a = __ffma2_rn(make_float2(x[64 * hh + 2 * i], x[64 * hh + 2 * i + 1]), sl2x2, nref2);
              const float p0 = ex2(a.x);
              const float p1 = ex2(a.y);
              sum4[i & 3] = __fadd2_rn(sum4[i & 3], make_float2(p0, p1));
              // P is rounded to 16 bits for the tensor core (half a step of the
              // inputs' type per weight); the row sum takes the unrounded values
              pk[i] = pack2<F16>(p0, p1);
            }
            tmem_st32(tP + 32u * hh, pk);
            if (kHalfP && hh == 0) {   // the first 64 keys' P: its half of P V may start
              tmem_st_wait();
              tc_fence_before();
              mbar_arrive_warp(bar(L::bPHalf + t));
            }
          }
          tmem_st_wait();
          const float2 s01 = __fadd2_rn(sum4[0], sum4[1]), s23 = __fadd2_rn(sum4[2], sum4[3]);
          const float2 s4 = __fadd2_rn(s01, s23);
          s_row = s4.x + s4.y;
          // (a row whose reference is still -inf, every earlier key masked,
          // always takes the row max)
          if (pass == 0 && __all_sync(0xFFFFFFFFu, s_row < kSpecSumLimit && m_ref != -INFINITY)) break;
        }
        l += s_row;
        tc_fence_before();
        mbar_arrive_warp(bar(L::bPFull + t));
        ++nS;
      }
      // O / l and the LSE, once the last PV has completed. A lane holds 32
      // columns of its row at a time, as four 16-byte chunks; transposed across
      // its quad it holds one chunk of four rows, and a quad writes 64 bytes of
      // each.
      if (ok) ok = bar_wait_warp(bar(L::bOFinal + t), nO & 1u, ctl, 324 + t);
      if (!ok) break;
      ++nO;
      tc_fence_after();
      // SPLIT: the first group joins what the second has, whose O it reads from TMEM:
      //   O = (2^(m0 - M) O_0 + 2^(m1 - M) O_1) / (2^(m0 - M) l_0 + 2^(m1 - M) l_1)
      float w0 = 1.f, w1 = 0.f;
      const bool join = SPLIT && w.has(1);
      if constexpr (SPLIT) {
        float2* stats = reinterpret_cast<float2*>(smem + L::kStats);
        if (join && t == 1) {
          stats[r] = make_float2(m_ref, l);
          tc_fence_before();
          mbar_arrive_warp(bar(L::bStats));
          ++nJ;
          continue;
        }
        if (join) {
          if (!(ok = bar_wait_warp(bar(L::bOFinal + 1), nJ & 1u, ctl, 325) &&
                     bar_wait_warp(bar(L::bStats), nJ & 1u, ctl, 329)))
            break;
          ++nJ;
          tc_fence_after();
          const float2 o1 = stats[r];
          const float M = fmaxf(m_ref, o1.x), ref = M == -INFINITY ? 0.f : M;
          w0 = ex2(m_ref - ref);
          w1 = ex2(o1.x - ref);
          l = fmaf(w0, l, w1 * o1.y);
          m_ref = M;
        }
      }
      const float inv_l = 1.f / l;
      const int s4 = lane & 3;
      const int row0 = kTile * qi + 32 * (warp & 3) + (lane & ~3);   // the quad's first row
      uint16_t* op = p.o + (int64_t)(w.start + row0) * p.o_tok + w.hq(t) * p.o_head + 8 * s4;
      uint32_t next[32];   // (the next columns come while these are written)
      tmem_ld32(tO, next);
#pragma unroll 1
      for (int cc = 0; cc < D / 32; ++cc) {
        uint32_t u[32];
        tmem_ld_wait(next);
#pragma unroll
        for (int i = 0; i < 32; ++i) u[i] = next[i];
        if (cc + 1 < D / 32) tmem_ld32(tO + 32u * (cc + 1), next);
        if constexpr (SPLIT) {
          if (join) {
            uint32_t u1[32];
            tmem_ld32(tO + (uint32_t)D + 32u * cc, u1);
            tmem_ld_wait(u1);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              u[i] = __float_as_uint(fmaf(w1, __uint_as_float(u1[i]), w0 * __uint_as_float(u[i])));
          }
        }
        uint32_t x[4][4];   // [word of a chunk][chunk of this row, then row of the quad]
#pragma unroll
        for (int wd = 0; wd < 4; ++wd) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            x[wd][j] = pack2<F16>(__uint_as_float(u[8 * j + 2 * wd]) * inv_l, __uint_as_float(u[8 * j + 2 * wd + 1]) * inv_l);
          quad_transpose(x[wd], (uint32_t)s4);
        }
        if (32 * cc + 8 * s4 < p.d) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (row0 + j < w.len)
              *reinterpret_cast<uint4*>(op + j * p.o_tok + 32 * cc) = make_uint4(x[0][j], x[1][j], x[2][j], x[3][j]);
        }
      }
      if (row < w.len)
        p.lse[(size_t)w.hq(t) * p.total + w.start + row] = (m_ref + log2f(l)) * 0.69314718055994531f;
      tc_fence_before();   // (the next PV of this tile waits for this group's next P)
      if (join) mbar_arrive_warp(bar(L::bJoined));
    }
  } else {
    regs_dec<kOtherRegs>();   // the last warp: no role
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0) report_aborted(ctl);
  if (warp == L::kOther + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool F16, int SLOTS, bool SPLIT, int SCORE>
cudaError_t launch_packed_fwd_d(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                const PackedFwdParams& p, cudaStream_t s) {
  using L = PackedFwdLayout<D, SPLIT, SCORE != kScorePlain>;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static PerDeviceOnce smem_set;
  e = once_per_device(smem_set, dev, [] {
    return cudaFuncSetAttribute(fa_packed_fwd_kernel<D, F16, SLOTS, SPLIT, SCORE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                L::kSmemBytes);
  });
  if (e != cudaSuccess) return e;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  PackedFwdParams q = p;
  // K and V of a key/value head (2 total d 16-bit elements) are re-read by the
  // items of its G query heads
  q.group = p.G / (p.Hq / p.heads) * l2_head_group(4.0 * p.total * p.d, p.Hq / p.G);
  // a CTA per item where items are taken by cancelling CTAs, else one per SM
  const long long most = (long long)p.cap_items * p.heads;
  return launch_pdl(true, fa_packed_fwd_kernel<D, F16, SLOTS, SPLIT, SCORE>, dim3((unsigned)(p.B <= kDirect || most < sms ? most : sms)),
                    dim3(L::kThreads), L::kSmemBytes, s, tq, tk, tv, q);
}

template <int SCORE>
cudaError_t launch_packed_fwd_score(bool f16, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                    const PackedFwdParams& p, cudaStream_t s) {
  auto run = [&](auto many, auto split) -> cudaError_t {
    constexpr int SLOTS = many ? kManySlots : 1;
    constexpr bool SPLIT = split;
    if (p.d <= 64)
      return f16 ? launch_packed_fwd_d<64, true, SLOTS, SPLIT, SCORE>(tq, tk, tv, p, s)
                 : launch_packed_fwd_d<64, false, SLOTS, SPLIT, SCORE>(tq, tk, tv, p, s);
    return f16 ? launch_packed_fwd_d<128, true, SLOTS, SPLIT, SCORE>(tq, tk, tv, p, s)
               : launch_packed_fwd_d<128, false, SLOTS, SPLIT, SCORE>(tq, tk, tv, p, s);
  };
  using Yes = std::true_type;
  using No = std::false_type;
  if (p.split) return run(No{}, Yes{});
  // (for scores of their own, lists of several slots serve every call: half as many kernels)
  if (SCORE != kScorePlain || packed_many(p.B)) return run(Yes{}, No{});
  if constexpr (SCORE == kScorePlain) return run(No{}, No{});
  return cudaErrorInvalidValue;
}

}  // namespace

}  // namespace fa
