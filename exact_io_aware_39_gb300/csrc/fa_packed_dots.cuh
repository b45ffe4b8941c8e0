// First pass of the packed backward for scores of their own (fa_packed_bwd.cuh):
// for every query row the dot D = rowsum(P * dP), with P recomputed from the LSE,
// dP = dO V^T, the LSE in log2 units, and a zeroed dQ accumulator.
//
// D is also rowsum(dO * O), which needs no products, but of the O that the
// forward rounded to 16 bits. Where a row has few keys of weight, dP - D is a small
// difference and that rounding shows: dQ and dK were off by 2.5e-3 of their norm
// in bf16 for scores of a standard deviation of 1, by 3.5e-3 to 5e-3 for 4 to 10, and
// by 6e-3 to 2e-2 in sequences of a few tokens; formed from P and dP in fp32 they
// are off by what rounding dS and the results makes.
//
// The roles are those of the forward (fa_packed_fwd.cuh): a work item is two
// query tiles that share the loads of K and V, two warpgroups for each (thread =
// row and half of its columns), which read S_t = Q_t K^T and dP_t = dO_t V^T from
// TMEM (four regions of 128 columns, all there are) and free each as soon as it is
// in registers, so that the tensor core works on the next one meanwhile.
// Bound: 4 d operations per visible pair on the tensor cores, and the scores'
// arithmetic. (32 / 8 heads, d = 128, capped: two sequences of 4547 and 5127 tokens
// 297 us, 1.30 PFLOP/s; 16 documents of 32-2048 tokens 81.) At 96 registers at
// launch 28-96 bytes a thread are spilled.
#pragma once

#include "fa_packed_rows.cuh"

namespace fa {

namespace {

template <int D>
struct PackedDotsLayout {
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kHalves = D / 64;
  static constexpr int kStages = D == 64 ? 8 : 3;               // K_e, V_e, K_(e+1), ...
  static constexpr int kQ = 0;                                  // [2] x (Q, dO)
  static constexpr int kKV = kQ + 4 * kTileBytes;
  static constexpr int kBar = kKV + kStages * kTileBytes;
  static constexpr int kItemRing = 4;
  static constexpr int bQFull = 0;                              // [2]
  static constexpr int bQEmpty = bQFull + 2;                    // [2]: the tile's last products are complete
  static constexpr int bFull = bQEmpty + 2;                     // [kStages]
  static constexpr int bEmpty = bFull + kStages;                // [kStages]
  static constexpr int bSFull = bEmpty + kStages;               // [2]
  static constexpr int bPFull = bSFull + 2;                     // [2]
  static constexpr int bSFree = bPFull + 2;                     // [2], 8 arrivals: S_t is in registers
  static constexpr int bPFree = bSFree + 2;                     // [2], 8: dP_t
  static constexpr int bItemFull = bPFree + 2;                  // [kItemRing]
  static constexpr int bItemEmpty = bItemFull + kItemRing;      // [kItemRing], 17: MMA and row warps
  static constexpr int bClc = bItemEmpty + kItemRing;
  static constexpr int bDrain = bClc + 1;
  static constexpr int kNumBars = bDrain + 1;
  static constexpr int kMisc = (kBar + 8 * kNumBars + 15) & ~15;   // tmem slot, abort flag, -, wait limit
  static constexpr int kRing = kMisc + 16;                      // [kItemRing] x {first row, length, unit or -1, head, first padded tile, -}
  static constexpr int kRingInts = 5;
  static constexpr int kClc = (kRing + 4 * kRingInts * kItemRing + 15) & ~15;
  static constexpr int kEx = kClc + 16;                         // [2] x [2] x [128] sums of a query tile's halves
  static constexpr int kSmemBytes = kEx + 4 * kTile * 4;
  static_assert(kSmemBytes <= 232448, "shared memory budget");
};

template <int D, bool F16, int SCORE>
__global__ void __launch_bounds__(kHalfThreads, 1)
fa_packed_dots_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                      const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap tdo,
                      const PackedBwdParams p, const int pair_heads, const int heads, const int group) {
  using L = PackedDotsLayout<D>;
  using Item = Pair<false, true>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x;
  const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);   // (the same in all lanes, as the compiler then knows)
  const int lane = tid & 31;
  auto bar = [&](int i) -> uint32_t { return sbase + L::kBar + 8u * (uint32_t)i; };
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  volatile uint32_t* abort_flag = misc + 1;
  volatile int* ring = reinterpret_cast<volatile int*>(smem + L::kRing);
  Ctl ctl{p.err, abort_flag};

  if ((sbase & 1023u) != 0u) {   // uniform across the CTA: nothing has started yet
    if (tid == 0) {
      uint32_t dummy = 0;
      Ctl c0{p.err, &dummy};
      report_error(c0, kErrSmemAlign, 385);
    }
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < L::kNumBars; ++i)
      mbar_init(bar(i), i >= L::bSFree && i < L::bPFree + 2 ? 8u
                        : i >= L::bItemEmpty && i < L::bItemEmpty + L::kItemRing ? 17u : 1u);
    abort_flag[0] = 0u;
    abort_flag[2] = p.wait_us;   // the wait limit, read by the slow path of every wait
    fence_mbar_init();
  }
  if (warp == 17) {
    tmem_alloc(smem_u32(misc), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();   // the barriers are initialised and TMEM allocated
  tc_fence_after();
  const uint32_t tmem = misc[0];
  grid_dep_wait();
  grid_dep_launch();

  // item k of this CTA from the ring (whole warps); w.c < 0 when none is left
  // or a wait failed (then it returns false)
  auto take_item = [&](int k, Item& w, int& slot0) -> bool {
    const int rs = k % L::kItemRing;
    w.c = -1;
    if (!bar_wait_warp(bar(L::bItemFull + rs), (uint32_t)(k / L::kItemRing) & 1u, ctl, 386)) return false;
    w.start = __shfl_sync(0xFFFFFFFFu, ring[L::kRingInts * rs], 0);
    w.len = __shfl_sync(0xFFFFFFFFu, ring[L::kRingInts * rs + 1], 0);
    w.c = __shfl_sync(0xFFFFFFFFu, ring[L::kRingInts * rs + 2], 0);
    w.head = __shfl_sync(0xFFFFFFFFu, ring[L::kRingInts * rs + 3], 0);
    slot0 = __shfl_sync(0xFFFFFFFFu, ring[L::kRingInts * rs + 4], 0);
    w.finish(pair_heads != 0, p.causal != 0);
    mbar_arrive_warp(bar(L::bItemEmpty + rs));
    return true;
  };

  if (warp == 16) {
    // ------------------------------------------------------------ items and loads
    regs_dec<kHalfOtherRegs>();
    if (lane == 0) {
      tma_prefetch_map(&tq);
      tma_prefetch_map(&tk);
      tma_prefetch_map(&tv);
      tma_prefetch_map(&tdo);
    }
    // up to kDirect sequences the list is made here and items are taken by
    // cancelling CTAs that have not started; else the plan's tiles are dealt out
    const bool direct = p.B <= kDirect;
    const int tiles = pair_heads ? 1 : 2;   // of a head, in an item
    DirectList<kManySlots, true> dl;
    int n_items = 0;
    if (direct) {
      dl.init(p.cu, p.score.prefix, p.B, p.total, kTile, p.cap_tiles, p.causal != 0, p.err, tiles);
      n_items = dl.items;
    } else {
      n_items = p.plan->tiles;
    }
    const int total = n_items * heads;
    int nl = 0;                  // K and V loads issued
    int nq0 = 0, nq1 = 0;        // Q and dO loads issued per query tile
    bool clc_out = false;
    uint32_t clc = 0u;
    bool ok = true;
    auto load = [&](const CUtensorMap* m, int hk, int row) -> bool {
      const int s = nl % L::kStages;
      if (nl >= L::kStages && !bar_wait_warp(bar(L::bEmpty + s), (uint32_t)(nl / L::kStages - 1) & 1u, ctl, 388)) return false;
      mbar_arrive_expect_tx_w(bar(L::bFull + s), L::kTileBytes);
      for (int a = 0; a < L::kHalves; ++a)
        tma_load_3d_w(sbase + L::kKV + s * L::kTileBytes + a * 16384, m, bar(L::bFull + s), 64 * a, hk, row);
      ++nl;
      return true;
    };
    int dealt = (int)blockIdx.x;
    for (int k = 0; ok; ++k) {
      const int rs = k % L::kItemRing;
      if (k >= L::kItemRing &&
          !(ok = bar_wait_warp(bar(L::bItemEmpty + rs), (uint32_t)(k / L::kItemRing - 1) & 1u, ctl, 387)))
        break;
      Item w;
      w.c = -1;
      int ring_c = -1, slot0 = 0;
      for (bool first = k == 0;; first = false) {
        int item = dealt;
        if (!direct) {
          dealt += (int)gridDim.x;
        } else if (!first) {
          if (lane == 0) {
            mbar_arrive_expect_tx(bar(L::bClc), 16u);
            clc_try_cancel(sbase + L::kClc, bar(L::bClc));
          }
          __syncwarp();
          clc_out = true;
          if (!(ok = bar_wait_warp(bar(L::bClc), clc & 1u, ctl, 389))) break;
          clc_out = false;
          ++clc;
          item = __shfl_sync(0xFFFFFFFFu, clc_first_ctaid_x(sbase + L::kClc), 0);
          if (item < 0) break;
          if (item >= total) continue;   // past the list: cancelled too, until none is left
        }
        if (item >= total) break;
        int head = 0;
        const int idx = split_grouped(item, group, n_items, heads, &head);
        PackedItem pi;
        if (direct) {
          pi = dl.at(idx, p.causal != 0);
          pi.c = with_prefix(pi.c, dl.prefix);
        } else {
          pi = p.tiles[idx];
          // (a sequence past the padded rows, of bounds that overlap, is left out)
          if (pi.slot0 + (pi.len + kTile - 1) / kTile > p.cap_tiles) continue;
          if (tiles == 2) {
            if (tile_of(pi.c) & 1) continue;   // (the second of a pair)
            pi.c = with_prefix(tile_of(pi.c) / 2, prefix_of(pi.c));
          }
        }
        w.start = __shfl_sync(0xFFFFFFFFu, pi.start, 0);
        w.len = __shfl_sync(0xFFFFFFFFu, pi.len, 0);
        ring_c = w.c = __shfl_sync(0xFFFFFFFFu, pi.c, 0);
        slot0 = __shfl_sync(0xFFFFFFFFu, pi.slot0, 0);
        w.head = head;
        w.finish(pair_heads != 0, p.causal != 0);
        break;
      }
      if (!ok) break;
      if (lane == 0) {
        ring[L::kRingInts * rs] = w.start;
        ring[L::kRingInts * rs + 1] = w.len;
        ring[L::kRingInts * rs + 2] = ring_c;
        ring[L::kRingInts * rs + 3] = w.head;
        ring[L::kRingInts * rs + 4] = slot0;
        mbar_arrive(bar(L::bItemFull + rs));   // (release: the ring entry is visible to the waiters)
      }
      if (w.c < 0) break;
      const int hk = w.hq(0) / p.G;
      if (k > 0)   // Q and dO wait for the item before: into L2 until then
#pragma unroll 1
        for (int t = 0; t < 2; ++t)
          for (int a = 0; w.has(t) && a < L::kHalves; ++a) {
            tma_prefetch_3d_w(&tq, 64 * a, w.hq(t), w.start + kTile * w.qi(t));
            tma_prefetch_3d_w(&tdo, 64 * a, w.hq(t), w.start + kTile * w.qi(t));
          }
#pragma unroll 1
      for (int e = 0; e < w.n && ok; ++e) {
        if (p.stall != 0u && e >= 1) { ok = false; break; }   // test of the timeout path: K of entry 1 never comes
        if (!(ok = load(&tk, hk, w.start + kTile * e))) break;
#pragma unroll 1
        for (int t = 0; e == 0 && t < 2 && ok; ++t) {
          if (!w.has(t)) continue;
          const int nt = t ? nq1 : nq0;
          if (nt > 0 && !(ok = bar_wait_warp(bar(L::bQEmpty + t), (uint32_t)(nt - 1) & 1u, ctl, 390))) break;
          mbar_arrive_expect_tx_w(bar(L::bQFull + t), 2u * L::kTileBytes);
          for (int a = 0; a < L::kHalves; ++a) {
            const uint32_t dst = sbase + L::kQ + 2 * t * L::kTileBytes + a * 16384;
            tma_load_3d_w(dst, &tq, bar(L::bQFull + t), 64 * a, w.hq(t), w.start + kTile * w.qi(t));
            tma_load_3d_w(dst + L::kTileBytes, &tdo, bar(L::bQFull + t), 64 * a, w.hq(t), w.start + kTile * w.qi(t));
          }
          (t ? nq1 : nq0) += 1;
        }
        if (ok) ok = load(&tv, hk, w.start + kTile * e);
      }
    }
    // every load and cancellation request issued has completed before the CTA exits
    if (lane == 0) {
      if (clc_out) drain_wait(bar(L::bClc), clc & 1u);
      if (nq0 > 0) drain_wait(bar(L::bQFull), (uint32_t)(nq0 - 1) & 1u);
      if (nq1 > 0) drain_wait(bar(L::bQFull + 1), (uint32_t)(nq1 - 1) & 1u);
#pragma unroll 1
      for (int s = 0; s < L::kStages && s < nl; ++s)
        drain_wait(bar(L::bFull + s), (uint32_t)((nl - 1 - s) / L::kStages) & 1u);
    }
  } else if (warp == 17) {
    // ------------------------------------------------------------ MMA issuer
    // (the whole warp runs the schedule, one elected lane issues): per entry e,
    // S_t = Q_t K_e^T for both query tiles, then dP_t = dO_t V_e^T, each once its
    // group has read the region's last contents
    regs_dec<kHalfOtherRegs>();
    constexpr uint32_t id = idesc_16<F16>(128, 128, false, false);
    const uint32_t dQ0 = desc_lo(desc_kmajor(sbase + L::kQ, 0));
    const uint32_t dKV0 = desc_lo(desc_kmajor(sbase + L::kKV, 0));
    constexpr uint32_t kSlotStep = (uint32_t)(L::kTileBytes >> 4);
    int nl = 0, nq[2] = {0, 0}, slot0 = 0;
    uint32_t ns[2] = {0u, 0u};      // entries of each query tile so far
    bool ok = true;
    Item w;
    for (int k = 0; ok && take_item(k, w, slot0) && w.c >= 0; ++k) {
      const int last[2] = {w.last(0), w.has(1) ? w.last(1) : -1};
#pragma unroll 1
      for (int e = 0; e < w.n && ok; ++e) {
#pragma unroll
        for (int which = 0; which < 2; ++which) {   // 0: S, 1: dP
          const int s = nl % L::kStages;
          if (!ok || !(ok = bar_wait_warp(bar(L::bFull + s), (uint32_t)(nl / L::kStages) & 1u, ctl, 391))) break;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (!ok || e > last[t]) continue;
            const int free_bar = (which == 0 ? L::bSFree : L::bPFree) + t;
            if (ns[t] > 0 && !(ok = bar_wait_warp(bar(free_bar), (ns[t] - 1u) & 1u, ctl, 392))) continue;
            if (which == 0 && e == 0 && !(ok = bar_wait_warp(bar(L::bQFull + t), (uint32_t)nq[t] & 1u, ctl, 393))) continue;
            tc_fence_after();
            const uint32_t a = dQ0 + (uint32_t)(2 * t + which) * kSlotStep, b = dKV0 + (uint32_t)s * kSlotStep;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
              mma_ss_lo(tmem + 128u * (uint32_t)t + 256u * (uint32_t)which, a + (uint32_t)kmajor_step(ks),
                        b + (uint32_t)kmajor_step(ks), id, ks > 0 ? 1u : 0u);
            mma_commit_w(bar((which == 0 ? L::bSFull : L::bPFull) + t));
            if (which == 1 && e == last[t]) mma_commit_w(bar(L::bQEmpty + t));   // Q_t and dO_t are no longer needed
            if (which == 1) ++ns[t];
          }
          if (ok) mma_commit_w(bar(L::bEmpty + s));
          ++nl;
        }
      }
      ++nq[0];
      nq[1] += w.has(1) ? 1 : 0;
    }
    // every MMA issued has completed before TMEM is freed
    mma_commit_w(bar(L::bDrain));
    drain_wait(bar(L::bDrain), 0);
  } else if (warp < 16) {
    // ------------------------------------------------------------ rows (thread = row and half of its columns)
    // The two groups of a query tile meet at the start and the end of an item, and
    // agree there whether all their waits held.
    regs_inc<kHalfRegs>();
    const int t = warp >> 3, h = (warp >> 2) & 1, r = tid & 127;
    const uint32_t pair_bar = 1u + (uint32_t)t;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + 128u * (uint32_t)t + 64u * (uint32_t)h + lane_off, tP = tS + 256u;
    volatile float* ex = reinterpret_cast<volatile float*>(smem + L::kEx) + 2 * kTile * t + r;
    uint32_t n = 0u;               // entries of this group so far
    int slot0 = 0;
    Item w;
    for (int k = 0;; ++k) {
      bool ok = take_item(k, w, slot0);
      ok = group_all(pair_bar, 256u, ok);
      if (!ok || w.c < 0) break;
      if (!w.has(t)) continue;
      const int qi = w.qi(t), last = w.last(t), hq = w.hq(t);
      const int row = kTile * qi + r;        // query index within the sequence
      const bool live = row < w.len;
      const size_t at = ((size_t)hq * p.cap_tiles + slot0 + qi) * kTile;   // the tile's first padded row
      const float lse2 = live ? p.lse[(size_t)hq * p.total + w.start + row] * 1.4426950408889634f : INFINITY;
      const float slope2 = p.score.slopes != nullptr ? p.score.slopes[hq] * 1.4426950408889634f : 0.f;
      {
        // the warp's rows of the dQ accumulator, every second piece (rows past the
        // sequence are added to as well, and never read)
        const int rows = min(32, w.len - (row - lane));
        float4* z = reinterpret_cast<float4*>(p.dq_acc + (at + r - lane) * p.d);
        for (int i = lane + 32 * h; i < rows * p.d / 4; i += 64) z[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
      float2 sum[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      for (int e = 0; e <= last; ++e, ++n) {
        if (!(ok = bar_wait_warp(bar(L::bSFull + t), n & 1u, ctl, 394))) break;
        tc_fence_after();
        uint32_t u[2][32];
        tmem_ld32(tS, u[0]);
        tmem_ld32(tS + 32u, u[1]);
        tmem_ld_wait(u[0]);
        tmem_ld_wait(u[1]);
        tc_fence_before();
        mbar_arrive_warp(bar(L::bSFree + t));
        // (as in the forward: keys from column `lim` on are masked)
        const bool partial = w.partial(e, qi);
        const int lim = (w.causal ? min(max(row + 1, w.pre), w.len) : w.len) - kTile * e - 64 * h;
        const ScoreTile st = score_tile<SCORE>(p.score, slope2, kTile * e + 64 * h, row, e < qi ? -1 : e > qi ? 1 : 0,
                                               e == qi && (!w.causal || w.pre > kTile * e), partial, lim, live);
        // Capped scores that are all within the polynomial's limit, without a bias or a mask, stay as they are
        // until the exponential: the polynomial beside it. (Two sequences of 4547 and 5127 tokens, 32 / 8 heads,
        // d = 128, forward and backward: 1669 -> 1640 us.)
        bool fast = false;
        if constexpr (SCORE == kScoreCap) {
          float most;
          const bool small = cap_vote(u, p.score, partial, lim, live, most);
          fast = small && !partial && !st.bias;
          if (!fast) {
            cap_args(u[0], p.score, partial, lim, small, -lse2);
            cap_args(u[1], p.score, partial, lim - 32, small, -lse2);
            if (st.bias) bias_args<SCORE>(u, p.scale_log2, st, -lse2);
          }
        } else {
          score_args<SCORE, false>(u, p.score, p.scale_log2, st, -lse2);
        }
        if (!(ok = bar_wait_warp(bar(L::bPFull + t), n & 1u, ctl, 395))) break;
        tc_fence_after();
        auto add = [&](auto polynomial) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t v[16];
            tmem_ld16(tP + 16u * c, v);
            if (c == 3) {
              tc_fence_before();
              mbar_arrive_warp(bar(L::bPFree + t));
            }
            if (!polynomial && partial) {   // (what lies past the sequence may be NaN)
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if (16 * c + i >= lim) v[i] = 0u;
            }
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              float2 a = pair_of(u[c >> 1], 16 * (c & 1) + i);
              if (polynomial) a = __ffma2_rn(a, cap_small_factor2(a, p.score), make_float2(-lse2, -lse2));
              sum[(i >> 1) & 3] = __ffma2_rn(make_float2(ex2(a.x), ex2(a.y)),
                                             make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), sum[(i >> 1) & 3]);
            }
          }
        };
        if (fast) add(std::true_type{});
        else add(std::false_type{});
      }
      const float2 s = __fadd2_rn(__fadd2_rn(sum[0], sum[1]), __fadd2_rn(sum[2], sum[3]));
      ex[kTile * h] = s.x + s.y;
      ok = group_all(pair_bar, 256u, ok);
      if (!ok) break;
      if (h == 0) {
        p.delta[at + r] = live ? ex[0] + ex[kTile] : 0.f;
        p.lse2[at + r] = lse2;
      }
    }
  } else {
    regs_dec<kHalfOtherRegs>();   // warps 18 and 19: no role
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0) report_aborted(ctl);
  if (warp == 17) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool F16, int SCORE>
cudaError_t launch_packed_dots(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& tdo,
                               const PackedBwdParams& p, int sms, cudaStream_t s) {
  using L = PackedDotsLayout<D>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static PerDeviceOnce smem_set;
  e = once_per_device(smem_set, dev, [] {
    return cudaFuncSetAttribute(fa_packed_dots_kernel<D, F16, SCORE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                L::kSmemBytes);
  });
  if (e != cudaSuccess) return e;
  const bool pair_heads = packed_pair_heads(p.Hq, p.Hk);
  const int heads = pair_heads ? p.Hq / 2 : p.Hq;
  const int group = p.G / (p.Hq / heads) * l2_head_group(4.0 * p.total * p.d, p.Hk);
  // a CTA per item where items are taken by cancelling CTAs, else one per SM
  const long long units = pair_heads ? p.cap_tiles : (long long)p.total / (2 * kTile) + p.B;
  const long long most = units * heads;
  return launch_pdl(false, fa_packed_dots_kernel<D, F16, SCORE>,
                    dim3((unsigned)(p.B <= kDirect ? most : (long long)p.cap_tiles * heads < sms ? (long long)p.cap_tiles * heads : sms)),
                    dim3(kHalfThreads), L::kSmemBytes, s, tq, tk, tv, tdo, p, (int)pair_heads, heads, group);
}

}  // namespace

}  // namespace fa
