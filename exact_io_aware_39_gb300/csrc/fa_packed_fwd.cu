// Forward pass over packed sequences with grouped heads, for sm_103a
// (tcgen05 tensor cores, TMEM accumulators, TMA staging).
//
// The computation of one pair of 128-row query tiles is that of fa_fwd.cu: a
// persistent CTA per SM with two softmax warpgroups (one per query tile), a TMA
// producer each for Q / K and for V, and one warp that runs the MMA schedule;
// S_t = Q_t K_j^T and O_t in TMEM, P_t packed to 16 bits into TMEM for the
// second product, the reference maximum moved only past 2^8. What is different:
//   * a work item is a pair of query tiles of one (sequence, query head). The
//     items of a call come from a list that the plan kernel makes on the device
//     (the lengths are there), heaviest first, and are taken from a counter;
//   * the tensors are [token, head, d] with any strides: a tile is a 3-D TMA
//     box of one head and 128 tokens. It may run into the next sequence: keys
//     past the end are masked in S, their rows of V are zeroed in shared memory
//     before the product (a zero weight times a NaN that lies there would be
//     NaN), and rows of O past the end are not stored (full groups of 32 rows
//     go out by TMA, the last one row by row);
//   * query head h reads key/value head h / G; neighbouring query heads run at
//     the same time, so a group's K and V come from L2 after their first read;
//   * the live key tiles of an item are a range, so no list is built.
//
// Bound: 4 d operations per visible pair on the tensor cores. At d = 128 each
// S tile costs a warpgroup 128 exponentials per row; the two query tiles
// alternate so that the products of one hide the softmax of the other.
#include "fa_packed.cuh"

namespace fa {

namespace {

constexpr int kFwdThreads = 384;
constexpr int kSoftmaxRegs = 216;   // 2 x 128 x 216 + 128 x 72 = 384 x 168 registers
constexpr int kOtherRegs = 72;
constexpr float kRescaleThreshold = 8.0f; // log2 units
constexpr float kSpecSumLimit = 256.0f;    // 2^kRescaleThreshold

template <int D>
struct PackedFwdLayout {
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kHalves = D / 64;
  // separate K and V rings; the K ring is the deeper one, since the S MMAs
  // that read K come first
  static constexpr int kStagesK = (D == 64) ? 5 : 3;
  static constexpr int kStagesV = (D == 64) ? 4 : 2;
  // Q buffers (each the two Q tiles of an item, and then the item's O
  // staging): at d = 64 two, so that the next item's Q and first K tiles are
  // loaded while this item runs; at d = 128 the shared memory holds one.
  // At d = 64, S_0, S_1 (128 columns each) and O_0, O_1 (64 each) leave 128
  // TMEM columns, which give each Q tile's P columns of their own: S_t is then
  // free as soon as its softmax group has read it into registers, and the
  // next S_t is computed while that group works on this one. At d = 128 the
  // four regions fill TMEM and P is packed over S in place.
  static constexpr bool kOwnP = (D == 64);
  static constexpr int kQBuf = (D == 64) ? 2 : 1;
  static constexpr int kQ = 0;
  static constexpr int kK = kQ + kQBuf * 2 * kTileBytes;
  static constexpr int kV = kK + kStagesK * kTileBytes;
  static constexpr int kBar = kV + kStagesV * kTileBytes;   // 8-byte mbarriers
  // barrier slots
  static constexpr int bQFull = 0;                    // [kQBuf]
  static constexpr int bKFull = bQFull + kQBuf;
  static constexpr int bKEmpty = bKFull + kStagesK;
  static constexpr int bVFull = bKEmpty + kStagesK;
  static constexpr int bVEmpty = bVFull + kStagesV;
  static constexpr int bSFull = bVEmpty + kStagesV;   // [2]
  static constexpr int bPFull = bSFull + 2;           // [2]
  static constexpr int bOFinal = bPFull + 2;          // [2]
  static constexpr int bSFree = bOFinal + 2;          // [2] S_t read into registers (own P columns only)
  static constexpr int bPVDone = bSFree + 2;          // [2] O_t += P_t V complete (own P columns only)
  static constexpr int bPHalf = bPVDone + 2;          // [2] P_t of the first 64 keys is in TMEM (P over S only)
  static constexpr int bDrain = bPHalf + 2;
  static constexpr int kNumBars = bDrain + 1;
  // 32-bit words: tmem slot, abort flag, -, wait limit, -, -, next item, -;
  // then per Q buffer b at 8 + 4 b the item: first row, length, pair, query head
  static constexpr int kMisc = kBar + 8 * kNumBars;
  static constexpr int kSmemBytes = kMisc + 4 * (8 + 4 * kQBuf);
  static_assert(kSmemBytes <= 232448, "shared memory budget");
};

// What the roles need of an item: its query tiles qi0 and qi0 + 1 (the second
// one may be missing), the key tiles 0 .. n - 1 live for either, the last one
// live for each, and per (key tile, query tile) whether it is live and masked.
struct Pair {
  int start, len, qi0, h;
  int n;
  bool two, causal;
  __device__ __forceinline__ Pair(const volatile uint32_t* m, int causal_)
      : start((int)m[0]), len((int)m[1]), qi0(2 * (int)m[2]), h((int)m[3]), causal(causal_ != 0) {
    const int nT = (len + kTile - 1) / kTile;
    two = qi0 + 1 < nT;
    n = causal ? min(nT, qi0 + 2) : nT;
  }
  __device__ __forceinline__ int last(int t) const { return t == 0 ? (causal ? qi0 : n - 1) : (two ? n - 1 : -1); }
  __device__ __forceinline__ bool live(int e, int t) const { return t == 0 ? (!causal || e <= qi0) : two; }
  __device__ __forceinline__ bool partial(int e, int t) const {
    return (causal && e == qi0 + t) || (e + 1) * kTile > len;
  }
  // valid rows of the last key tile when it is not full, else 0
  __device__ __forceinline__ int tail() const { return len & (kTile - 1); }
};

template <int D, bool F16>
__global__ void __launch_bounds__(kFwdThreads, 1)
fa_packed_fwd_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
              const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap to,
              const PackedFwdParams p) {
  using L = PackedFwdLayout<D>;
  // With P over S (d = 128), P of a tile's first 64 keys goes to the tensor
  // core before the rest is formed, and its half of P V runs meanwhile; the
  // softmax then always takes the row max first, since P may not be formed
  // again once half of it has been used
  constexpr bool kHalfP = !L::kOwnP;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);

  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;

  auto bar = [&](int i) -> uint32_t { return sbase + L::kBar + 8u * (uint32_t)i; };
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  volatile uint32_t* abort_flag = misc + 1;
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
    for (int i = 0; i < L::kNumBars; ++i)
      mbar_init(bar(i), (i == L::bPFull || i == L::bPFull + 1 || i == L::bSFree || i == L::bSFree + 1 ||
                         i == L::bPHalf || i == L::bPHalf + 1) ? 4u : 1u);   // 4 = warps
    abort_flag[0] = 0u;
    abort_flag[2] = p.wait_us;   // the wait limit, read by the slow path of every wait
    fence_mbar_init();
  }
  if (warp == 9) {
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

  // Persistent over items: the first is this CTA's own, each further one the
  // next of a counter that the plan kernel zeroed. The work order walks groups
  // of p.group query heads whose K and V fit in L2 together, within a group
  // the items heaviest first, and for each item the heads of the group. Every
  // ring and barrier phase runs on across items: eK / eV count the K / V ring
  // entries of the items before this one, and each role keeps its own counts.
  const int n_items = p.plan->items;
  const int total = n_items * p.Hq;
  int eK = 0, eV = 0;
  int nk = 0, nv = 0;                     // K / V loads issued (producer threads)
  uint32_t ns[2] = {0u, 0u}, npv[2] = {0u, 0u};   // S and PV groups issued per Q tile (MMA warp)
  uint32_t nS = 0u, nOF = 0u;             // S tiles and final O read by this softmax group
  int item = (int)blockIdx.x;
  uint32_t kq = 0u;                       // items started: the phase of the Q barrier
  // The roles meet at a named barrier before each item (its description is in
  // shared memory) and after it (its O is stored, its products read out).
  auto item_sync = [&]() {
    tc_fence_before();
    named_bar_sync(1, kFwdThreads);
    tc_fence_after();
  };
  // after an item: the next one, or none (then every role leaves its loop)
  auto next_item = [&]() -> int {
    const int next = (int)misc[6];
    return abort_flag[0] != 0u ? -1 : next;
  };
  if (item >= total) {
    // nothing for this CTA (uniform)
  } else if (warp == 8) {
    regs_dec<kOtherRegs>();
    uint32_t nq[2] = {0u, 0u};   // Q loads issued into each buffer (lane 0)
    // K of key tile e of item w into ring entry n, once the MMAs of the entry
    // that used the slot before (of this item or an earlier one) have read it
    auto load_k = [&](const Pair& w, int e, int n) -> bool {
      const int sk = n % L::kStagesK;
      if (n >= L::kStagesK && !mbar_wait(bar(L::bKEmpty + sk), (uint32_t)(n / L::kStagesK - 1) & 1u, ctl, 311))
        return false;
      mbar_arrive_expect_tx(bar(L::bKFull + sk), L::kTileBytes);
      for (int h = 0; h < L::kHalves; ++h)
        tma_load_3d(sbase + L::kK + sk * L::kTileBytes + h * 16384, &tk, bar(L::bKFull + sk), 64 * h, w.h / p.G,
                    w.start + kTile * e);
      ++nk;
      return true;
    };
    // Sets item `it` up in buffer qb (lane 0): its description is written down,
    // its Q tiles are loaded, and the first ring's worth of its K tiles (ring
    // entries base, base + 1, ...). Returns the K loads issued.
    auto setup = [&](int it, int qb, int base) -> int {
      int kpre = 0;
      if (lane == 0) {
        int h = 0;
        const PackedItem pi = p.items[split_grouped(it, p.group, n_items, p.Hq, &h)];
        uint32_t* m = misc + 8 + 4 * qb;
        m[0] = (uint32_t)pi.start;
        m[1] = (uint32_t)pi.len;
        m[2] = (uint32_t)pi.c;
        m[3] = (uint32_t)h;
        const Pair w(m, p.causal);
        mbar_arrive_expect_tx(bar(L::bQFull + qb), (w.two ? 2u : 1u) * L::kTileBytes);
        for (int t = 0; t < (w.two ? 2 : 1); ++t)
          for (int a = 0; a < L::kHalves; ++a)
            tma_load_3d(sbase + L::kQ + (2 * qb + t) * L::kTileBytes + a * 16384, &tq, bar(L::bQFull + qb), 64 * a, h,
                        w.start + kTile * (w.qi0 + t));
        ++nq[qb];
        for (; kpre < w.n && kpre < L::kStagesK; ++kpre) {
          if (p.stall != 0u && kpre >= 1) break;   // test of the timeout path: K of entry 1 never comes
          if (!load_k(w, kpre, base + kpre)) break;
        }
      }
      return kpre;
    };
    if (lane == 0) {
      tma_prefetch_map(&tq);
      tma_prefetch_map(&tk);
    }
    int kpre = setup(item, 0, 0);   // K loads of the current item issued during its set-up (lane 0)
    for (;; ++kq) {
      const int qb = (int)(kq % L::kQBuf);
      item_sync();
      // ------------------------------------------------------------ Q and K producer
      const Pair w(misc + 8 + 4 * qb, p.causal);
      int next = -1;
      if (lane == 0) {
        bool ok = true;
        for (int e = kpre; e < w.n && ok; ++e) {
          if (p.stall != 0u && e >= 1) ok = false;   // test of the timeout path: K of entry 1 never comes
          else ok = load_k(w, e, eK + e);
        }
        // every K load of the item is issued: take the next item
        if (ok) {
          next = (int)gridDim.x + (int)atomicAdd(&p.plan->sched, 1u);
          if (next >= total) next = -1;
        }
        misc[6] = (uint32_t)next;
      }
      // with two buffers the next item is set up while this one runs (the
      // other buffer's item has been stored: every role has passed the barrier
      // after it)
      next = __shfl_sync(0xFFFFFFFFu, next, 0);
      if (L::kQBuf == 2 && next >= 0) kpre = setup(next, qb ^ 1, eK + w.n);
      item_sync();
      item = next_item();
      if (item < 0) break;
      eK += w.n;
      if (L::kQBuf == 1) kpre = setup(item, 0, eK);
    }
    // every load issued has completed before the CTA exits; loads were issued
    // in ring order, so the last load into slot
    // s was number s + S * floor((n - 1 - s) / S)
    if (lane == 0) {
      for (int b = 0; b < L::kQBuf; ++b)
        if (nq[b] > 0u) drain_wait(bar(L::bQFull + b), (nq[b] - 1u) & 1u);
      for (int s = 0; s < L::kStagesK && s < nk; ++s)
        drain_wait(bar(L::bKFull + s), (uint32_t)((nk - 1 - s) / L::kStagesK) & 1u);
    }
  } else if (warp == 10) {
    regs_dec<kOtherRegs>();
    for (;; ++kq) {
      const int qb = (int)(kq % L::kQBuf);
      item_sync();
      const Pair w(misc + 8 + 4 * qb, p.causal);
      // ------------------------------------------------------------ V producer
      // (its own thread, so that the K ring can run ahead of the V ring)
      if (lane == 0) {
        if (kq == 0u) tma_prefetch_map(&tv);
        for (int e = 0; e < w.n; ++e) {
          const int n = eV + e;
          const int sv = n % L::kStagesV;
          if (n >= L::kStagesV && !mbar_wait(bar(L::bVEmpty + sv), (uint32_t)(n / L::kStagesV - 1) & 1u, ctl, 312))
            break;
          mbar_arrive_expect_tx(bar(L::bVFull + sv), L::kTileBytes);
          for (int h = 0; h < L::kHalves; ++h)
            tma_load_3d(sbase + L::kV + sv * L::kTileBytes + h * 16384, &tv, bar(L::bVFull + sv),
                        64 * h, w.h / p.G, w.start + kTile * e);
          ++nv;
        }
      }
      item_sync();
      item = next_item();
      if (item < 0) break;
      eV += w.n;
    }
    if (lane == 0)
      for (int s = 0; s < L::kStagesV && s < nv; ++s)
        drain_wait(bar(L::bVFull + s), (uint32_t)((nv - 1 - s) / L::kStagesV) & 1u);
  } else if (warp == 9) {
    regs_dec<kOtherRegs>();
    for (;; ++kq) {
      const int qb = (int)(kq % L::kQBuf);
      item_sync();
      const Pair w(misc + 8 + 4 * qb, p.causal);
      const int len = w.n;
      // ------------------------------------------------------------ MMA issuer
      // Fixed schedule over the live key tiles: at entry e, for each Q tile t, first
      // the pending O_t += P_t V of t's previous live entry (waiting for P_t),
      // then S_t = Q_t K_e^T if t is live at e. For dense rows this is
      //   PV0(e-1), S0(e), PV1(e-1), S1(e), PV0(e), ...
      // so that while one softmax group works the tensor core runs the other
      // tile's products. A pending PV is issued at the very next entry, so each
      // V slot is released one entry after its load and the K slot of entry e
      // right after its S products.
      {   // the whole warp runs the schedule; one elected lane issues each MMA and commit
        constexpr uint32_t idS = idesc_16<F16>(128, 128, false, false);
        constexpr uint32_t idO = idesc_16<F16>(128, D, false, true);
        const uint32_t tS[2] = {tmem + 0u, tmem + 128u};
        const uint32_t tO[2] = {tmem + 256u, tmem + 256u + (uint32_t)D};
        // P_t: over S_t, or in columns of its own (after O_1)
        const uint32_t tP[2] = {L::kOwnP ? tmem + 256u + 2u * D : tS[0], L::kOwnP ? tmem + 320u + 2u * D : tS[1]};
        const uint64_t dQ[2] = {desc_kmajor(sbase + L::kQ + 2 * qb * L::kTileBytes, 0),
                                desc_kmajor(sbase + L::kQ + (2 * qb + 1) * L::kTileBytes, 0)};
        const uint64_t dK0 = desc_kmajor(sbase + L::kK, 0);
        const uint64_t dV0 = desc_mnmajor(sbase + L::kV, 0);
        constexpr uint64_t kSlotStep = (uint64_t)(L::kTileBytes >> 4);
        int prev[2] = {-1, -1};       // entry of the pending PV of each Q tile
        // the last entry live for each Q tile: its PV completes O_t, which the
        // softmax group may then read out while the other tile's products run
        const int lastE[2] = {w.last(0), w.last(1)};
        uint32_t npv_item[2] = {0u, 0u};   // PV groups of this item per Q tile
        // the rows of V behind the sequence's end are zeroed once, before the
        // first product that reads the last key tile
        int tail_entry = w.tail() != 0 ? (w.len + kTile - 1) / kTile - 1 : -1;
        bool ok = mbar_wait_warp(bar(L::bQFull + qb), (kq / L::kQBuf) & 1u, ctl, 314);
        tc_fence_after();

        // O_t += P_t V_{entry pe}
        auto issue_pv = [&](int t, int pe) -> bool {
          const int nvp = eV + pe;
          const int sv = nvp % L::kStagesV;
          if (!mbar_wait_warp(bar((kHalfP ? L::bPHalf : L::bPFull) + t), npv[t] & 1u, ctl, 315)) return false;
          if (!mbar_wait_warp(bar(L::bVFull + sv), (uint32_t)(nvp / L::kStagesV) & 1u, ctl, 316)) return false;
          if (pe == tail_entry) {
            zero_tail_rows<D>(smem + L::kV + sv * L::kTileBytes, w.tail());
            tail_entry = -1;
          }
          tc_fence_after();
          const uint64_t dV = dV0 + (uint64_t)sv * kSlotStep;
          const uint32_t acc0 = npv_item[t] > 0 ? 1u : 0u;
#pragma unroll
          for (int ks = 0; ks < kTile / 16; ++ks) {
            if (kHalfP && ks == kTile / 32) {   // the second half of P
              if (!mbar_wait_warp(bar(L::bPFull + t), npv[t] & 1u, ctl, 315)) return false;
              tc_fence_after();
            }
            mma_ts_w(tO[t], tP[t] + (uint32_t)ks * 8u, dV + mnmajor_step(ks), idO, ks > 0 ? 1u : acc0);
          }
          if constexpr (L::kOwnP) mma_commit_w(bar(L::bPVDone + t));   // P_t may be rewritten, O_t rescaled
          if (pe == lastE[t]) mma_commit_w(bar(L::bOFinal + t));       // O_t is complete
          ++npv[t];
          ++npv_item[t];
          return true;
        };

        if constexpr (L::kOwnP) {
          // Own P columns: at entry e, first S_t(e) for each live tile, each as
          // soon as group t has read its previous S_t into registers, then the
          // PVs of entry e - 1. For dense rows:
          //   S0(e), S1(e), PV0(e-1), PV1(e-1), S0(e+1), ...
          // so S_t(e+1) is computed while group t still works on S_t(e).
          for (int e = 0; e < len && ok; ++e) {
            const int sk = (eK + e) % L::kStagesK;
            bool k_ready = false;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if (!ok || !w.live(e, t)) continue;
              if (ns[t] > 0 && !(ok = mbar_wait_warp(bar(L::bSFree + t), (ns[t] - 1u) & 1u, ctl, 318))) break;
              if (!k_ready) {
                ok = mbar_wait_warp(bar(L::bKFull + sk), (uint32_t)((eK + e) / L::kStagesK) & 1u, ctl, 317);
                if (!ok) break;
                tc_fence_after();
                k_ready = true;
              }
              const uint64_t dK = dK0 + (uint64_t)sk * kSlotStep;
#pragma unroll
              for (int ks = 0; ks < D / 16; ++ks)
                mma_ss_w(tS[t], dQ[t] + kmajor_step(ks), dK + kmajor_step(ks), idS, ks > 0 ? 1u : 0u);
              mma_commit_w(bar(L::bSFull + t));
              ++ns[t];
            }
            if (!ok) break;
            mma_commit_w(bar(L::bKEmpty + sk));   // K_e is no longer needed
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if (ok && prev[t] >= 0) ok = issue_pv(t, prev[t]);
              prev[t] = w.live(e, t) ? e : -1;
            }
            if (!ok) break;
            if (e > 0) mma_commit_w(bar(L::bVEmpty + (eV + e - 1) % L::kStagesV));   // both PVs of entry e-1 issued
          }
        } else {
          for (int e = 0; e < len && ok; ++e) {
            const int sk = (eK + e) % L::kStagesK;
            bool k_ready = false;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if (!ok) break;
              if (prev[t] >= 0) {
                ok = issue_pv(t, prev[t]);
                prev[t] = -1;
                if (!ok) break;
              }
              if (w.live(e, t)) {
                if (!k_ready) {
                  ok = mbar_wait_warp(bar(L::bKFull + sk), (uint32_t)((eK + e) / L::kStagesK) & 1u, ctl, 317);
                  if (!ok) break;
                  tc_fence_after();
                  k_ready = true;
                }
                const uint64_t dK = dK0 + (uint64_t)sk * kSlotStep;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                  mma_ss_w(tS[t], dQ[t] + kmajor_step(ks), dK + kmajor_step(ks), idS, ks > 0 ? 1u : 0u);
                mma_commit_w(bar(L::bSFull + t));
                prev[t] = e;
              }
            }
            if (!ok) break;
            mma_commit_w(bar(L::bKEmpty + sk));                       // K_e is no longer needed
            if (e > 0) mma_commit_w(bar(L::bVEmpty + (eV + e - 1) % L::kStagesV));   // both PVs of entry e-1 issued
          }
        }
        if (ok) {
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (ok && prev[t] >= 0) ok = issue_pv(t, prev[t]);   // (commits O_t's completion)
          }
          // the last entry's V slot goes back to the producer
          if (ok && len > 0) mma_commit_w(bar(L::bVEmpty + (eV + len - 1) % L::kStagesV));
        }
      }
      item_sync();
      item = next_item();
      if (item < 0) break;
      eK += len;
      eV += len;
    }
    // every MMA issued has completed before TMEM is freed
    mma_commit_w(bar(L::bDrain));
    drain_wait(bar(L::bDrain), 0);
  } else if (warp < 8) {
    regs_inc<kSoftmaxRegs>();
    for (;; ++kq) {
      item_sync();
      const int qb = (int)(kq % L::kQBuf);
      const Pair w(misc + 8 + 4 * qb, p.causal);
      const int len = w.n, qi0 = w.qi0;
      // ------------------------------------------------------------ softmax groups
      const int t = warp >> 2;                 // Q tile of this warpgroup
      const int r = tid & 127;                 // row within the tile = TMEM lane
      const int qi = qi0 + t;
      const int row = kTile * qi + r;          // query index within the sequence
      const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
      const uint32_t tS = tmem + (uint32_t)(t * 128) + lane_off;
      const uint32_t tO = tmem + 256u + (uint32_t)(t * D) + lane_off;
      const uint32_t tP = L::kOwnP ? tmem + 256u + 2u * D + 64u * (uint32_t)t + lane_off : tS;
      const float sl2 = p.scale_log2;

      float m_ref = -INFINITY;
      float l = 0.f;
      uint32_t n = 0;   // S tiles of this item (nS: of all items)
      const bool has = t == 0 || w.two;        // this query tile exists
      bool ok = has;
      for (int e = 0; e < len && ok; ++e) {
        if (!w.live(e, t)) continue;
        if (!mbar_wait_warp(bar(L::bSFull + t), nS & 1u, ctl, 320 + t)) { ok = false; break; }
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
        if (w.partial(e, t)) {
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
          if (!mbar_wait_warp(bar(L::bPVDone + t), (nS - 1u) & 1u, ctl, 326 + t)) { ok = false; break; }
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
        ++n;
        ++nS;
      }

      if (has) {
        // all MMAs that read Q_t have completed (or never ran); make sure the
        // Q load itself has landed before its buffer is reused for staging O
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (ok) ok = mbar_wait_warp(bar(L::bQFull + qb), (kq / L::kQBuf) & 1u, ctl, 322 + t);
        if (ok && n > 0) ok = mbar_wait_warp(bar(L::bOFinal + t), nOF & 1u, ctl, 324 + t);
        if (n > 0) ++nOF;
        if (!ok) drain_wait(bar(L::bQFull + qb), (kq / L::kQBuf) & 1u);   // after an abort: the Q load (always issued) lands before its buffer is rewritten
        tc_fence_after();
        uint8_t* stage = smem + L::kQ + (2 * qb + t) * L::kTileBytes;
        const float inv_l = n > 0 ? 1.f / l : 0.f;
        const bool have_o = ok && n > 0;
#pragma unroll
        for (int cc = 0; cc < D / 32; ++cc) {
          uint32_t u[32];
          if (have_o) {
            tmem_ld32(tO + 32u * cc, u);
            tmem_ld_wait(u);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) u[i] = 0u;
          }
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i)
            pk[i] = pack2<F16>(__uint_as_float(u[2 * i]) * inv_l, __uint_as_float(u[2 * i + 1]) * inv_l);
          // 32 columns = 4 chunks of 16 bytes, 128B-swizzled rows
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int col = 32 * cc + 8 * k;           // first column of the chunk
            const int h = col >> 6;                    // 64-column half
            const int chunk = (col & 63) >> 3;         // chunk within the 128-byte row
            uint8_t* dst = stage + h * 16384 + (r >> 3) * 1024 + (r & 7) * 128 + ((chunk ^ (r & 7)) << 4);
            *reinterpret_cast<uint4*>(dst) = make_uint4(pk[4 * k], pk[4 * k + 1], pk[4 * k + 2], pk[4 * k + 3]);
          }
        }
        if (row < w.len)
          p.lse[(size_t)w.h * p.total + w.start + row] = (m_ref + log2f(l)) * 0.69314718055994531f;
        // each warp stores its own 32 rows, so that no warp ever waits for
        // another at a group-wide barrier: all 32 by TMA, or, where the sequence
        // ends among them, the rows up to its end
        fence_proxy_async_smem();
        __syncwarp();
        const int row0 = kTile * qi + 32 * (warp & 3);
        const int rows = min(32, w.len - row0);
        if (rows == 32) {
          if (lane == 0) {
            for (int h = 0; h < L::kHalves; ++h)
              tma_store_3d(&to, smem_u32(stage) + h * 16384 + 4096 * (warp & 3), 64 * h, w.h, w.start + row0);
            bulk_commit_group();
            bulk_wait_group_read_all();   // the store has read the staging; the grid's end makes it visible
          }
        } else if (rows > 0) {
          uint16_t* op = p.o + (int64_t)(w.start + row0) * p.o_tok + w.h * p.o_head;
          const int chunks = p.d >> 3;
          for (int i = lane; i < rows * chunks; i += 32) {
            const int rr = i / chunks, ch = i % chunks;
            *reinterpret_cast<uint4*>(op + rr * p.o_tok + 8 * ch) =
                *reinterpret_cast<const uint4*>(stage + tile_chunk(32 * (warp & 3) + rr, ch));
          }
          fence_proxy_async_smem();   // read before TMA writes the buffer again
        }
      }
      item_sync();
      item = next_item();
      if (item < 0) break;
    }
  } else {
    regs_dec<kOtherRegs>();   // warp 11: no role of its own, it only keeps the item barriers
    for (;; ++kq) {
      item_sync();
      item_sync();
      item = next_item();
      if (item < 0) break;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool F16>
cudaError_t launch_packed_fwd_d(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                const CUtensorMap& to, const PackedFwdParams& p, cudaStream_t s) {
  using L = PackedFwdLayout<D>;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static PerDeviceOnce smem_set;
  e = once_per_device(smem_set, dev, [] {
    return cudaFuncSetAttribute(fa_packed_fwd_kernel<D, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                L::kSmemBytes);
  });
  if (e != cudaSuccess) return e;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  PackedFwdParams q = p;
  // K and V of a key/value head (2 total d 16-bit elements) are re-read by the
  // items of its G query heads
  q.group = p.G * l2_head_group(4.0 * p.total * p.d, p.Hq / p.G);
  const long long most = (long long)p.cap_items * p.Hq;
  return launch_pdl(true, fa_packed_fwd_kernel<D, F16>, dim3((unsigned)(most < sms ? most : sms)), dim3(kFwdThreads),
                    L::kSmemBytes, s, tq, tk, tv, to, q);
}

}  // namespace

cudaError_t launch_packed_fwd(bool f16, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                              const CUtensorMap& to, const PackedFwdParams& p, cudaStream_t s) {
  if (p.d <= 64)
    return f16 ? launch_packed_fwd_d<64, true>(tq, tk, tv, to, p, s) : launch_packed_fwd_d<64, false>(tq, tk, tv, to, p, s);
  return f16 ? launch_packed_fwd_d<128, true>(tq, tk, tv, to, p, s) : launch_packed_fwd_d<128, false>(tq, tk, tv, to, p, s);
}

}  // namespace fa
