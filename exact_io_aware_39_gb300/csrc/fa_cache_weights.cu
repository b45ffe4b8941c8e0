// The attention that cached keys receive from the newest tokens, for sm_103a
// (flash_attn_cached_weights in flash_attn_scored.h):
//   w_j = past_j + sum over the Nq tokens i and the G query heads of a key/value
//         head of exp(u_ij - LSE_i).
//
// The LSE is known, so a tile of keys needs nothing of the others: no running
// maximum, no join. Reading the keys is the work, 2 d bytes for 2 d Nq G
// operations, and the layout is that of the attention (fa_cached.cuh): the key
// tiles of all (sequence, key/value head) pairs are cut into equal ranges, one
// for each warp, which loads them by TMA into a ring of its own and multiplies
// with mma.sync. A tile's keys go to registers as the products' second operand,
// and its place in the ring is loaded again; the weights are summed over the rows
// in fp32 in a fixed order, and each key's sum is written by one lane, so results
// repeat. More than 16 query rows go to a kernel of their own (below).
//
// The 16 bytes a lane reads of a key are 8 neighbouring dims (16 in e4m3), which
// it spreads over two (four) K steps of the product; the queries are read in the
// same order, so that a lane reads them by 16 bytes as well.
#include "fa_cached.cuh"

namespace fa {

namespace {

struct WeightsParams {
  CachedParams c;       // (q .. lens, err, sizes, score; o and the parts are not used)
  const float* rows_lse;  // [B, Hq, Nq]
  const float* past;    // [num_pages, Hk, page_size] or null
  float* w;             // the same
};

template <int D, bool E4M3>
struct WeightsLayout {
  static constexpr int kWarps = 12;
  static constexpr int kKT = 4096 / D;                          // keys of a tile: 64 registers of fragments
  static constexpr int kRowBytes = E4M3 ? D : 128;              // of a swizzle atom
  static constexpr int kAtoms = E4M3 ? 1 : D / 64;
  static constexpr int kAtomBytes = kKT * kRowBytes;
  static constexpr int kStageBytes = kAtoms * kAtomBytes;       // 8 KB, 4 in e4m3
  static constexpr int kStages = 16384 / kStageBytes;
  static constexpr int kWarpBytes = kStages * kStageBytes;
  static constexpr int kScaleBytes = E4M3 ? 8 * kKT : 0;
  static constexpr int kScale = kWarps * kWarpBytes;
  static constexpr int kBar = kScale + kWarps * kStages * kScaleBytes;
  static constexpr int kMisc = kBar + 8 * kWarps * kStages;     // abort flag, -, wait limit, -
  static constexpr int kScan = kMisc + 16;                      // int64 [kWarps] totals, int64 [kWarps] starts, int [kWarps]
  static constexpr int kSmemBytes = (kScan + kWarps * 20 + 15) & ~15;
  static constexpr uint32_t kTxBytes = kStageBytes + (E4M3 ? kKT * 4u : 0u);
  static_assert(kSmemBytes <= 232448, "shared memory budget");
};

// Sums over the lanes of a column (g), halving what each lane keeps: bit 2 of g with
// the upper bit of n, and so on. v: [NT keys of 8][2]; the sums of this lane's keys
// end in v[0] (and, of 64 keys, v[1]).
template <int NT>
__device__ __forceinline__ void column_sums(float (&v)[2 * NT], int g) {
#pragma unroll
  for (int b = 0; b < 3; ++b) {
    const int half = NT >> b;             // values kept: NT, NT / 2, NT / 4
    const bool up = (g >> (2 - b)) & 1;
#pragma unroll
    for (int x = 0; x < half; ++x) {
      const float give = up ? v[x] : v[half + x], keep = up ? v[half + x] : v[x];
      v[x] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, 16 >> b);
    }
  }
}

template <int D, bool E4M3, bool F16>
__global__ void __launch_bounds__(32 * WeightsLayout<D, E4M3>::kWarps, 1)
fa_cache_weights_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tks,
                        const WeightsParams wp) {
  using L = WeightsLayout<D, E4M3>;
  constexpr int KT = L::kKT, NT = KT / 8, kWarps = L::kWarps, kSteps = D / 16;
  const CachedParams& p = wp.c;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  auto same = [](int v) -> int { return __shfl_sync(0xFFFFFFFFu, v, 0); };   // (known to be the same in all lanes)
  const int tid = threadIdx.x, warp = same(tid >> 5), lane = tid & 31;
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  volatile uint32_t* abort_flag = misc;
  Ctl ctl{p.err, abort_flag};
  if ((sbase & 1023u) != 0u) {   // uniform across the CTA: nothing has started yet
    if (tid == 0) {
      uint32_t dummy = 0;
      Ctl c0{p.err, &dummy};
      report_error(c0, kErrSmemAlign, 210);
    }
    return;
  }
  auto bar = [&](int s) -> uint32_t { return sbase + L::kBar + 8u * (uint32_t)(warp * L::kStages + s); };
  if (lane == 0)
    for (int s = 0; s < L::kStages; ++s) mbar_init(bar(s), 1u);
  if (tid == 0) {
    misc[0] = 0u;
    misc[2] = p.wait_us;
  }
  fence_mbar_init();
  grid_dep_wait();   // global memory is read and written only from here on

  // ---- this warp's range of the tiles of all sequences, for each the heads one
  // after another
  const int cap = p.max_pages << p.ps_log2;
  auto seq_len = [&](int b) -> int {
    const int n = p.lens[b];
    return n < 0 ? 0 : (n > cap ? cap : n);
  };
  auto tiles_of = [&](int len) -> int { return (len + KT - 1) / KT; };
  struct At {
    int b, hk, j, n, len;
  } w0;
  long long* tot = reinterpret_cast<long long*>(smem + L::kScan);
  long long* start_t = tot + kWarps;      // first tile of each warp's range, then the tiles of the sequences before it
  int* start_b = reinterpret_cast<int*>(start_t + kWarps);
  const int per = (p.B + 32 * kWarps - 1) / (32 * kWarps);
  const int b_lo = min(p.B, tid * per), b_hi = min(p.B, b_lo + per);
  long long mine = 0;
  for (int b = b_lo; b < b_hi; ++b) mine += tiles_of(seq_len(b));
  long long incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long o = __shfl_up_sync(0xFFFFFFFFu, incl, off);
    if (lane >= off) incl += o;
  }
  if (lane == 31) tot[warp] = incl;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += tot[w];
    all += tot[w];
  }
  const long long total = all * p.Hk;
  const int workers = (int)min((long long)(kWarps * gridDim.x), total);
  const int me = warp * (int)gridDim.x + (int)blockIdx.x;   // (neighbouring ranges go to different SMs)
  auto range_start = [&](int w) -> long long { return total * w / workers; };
  const long long t0 = me < workers ? range_start(me) : total;
  if (lane == 0) start_t[warp] = t0;
  __syncthreads();
  long long cum = before + incl - mine;   // tiles of the sequences before b_lo
  for (int b = b_lo; b < b_hi; ++b) {
    const long long lo = cum * p.Hk, hi = (cum += tiles_of(seq_len(b))) * p.Hk;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      if (start_t[w] >= lo && start_t[w] < hi) {
        start_b[w] = b;
        tot[w] = lo;
      }
  }
  __syncthreads();
  grid_dep_launch();
  if (me >= workers) return;
  const int todo = same((int)(range_start(me + 1) - t0));
  w0.b = same(start_b[warp]);
  w0.len = same(seq_len(w0.b));
  w0.n = tiles_of(w0.len);
  const long long rem = t0 - tot[warp];
  w0.hk = same((int)(rem / w0.n));
  w0.j = same((int)(rem % w0.n));
  auto advance = [&](At& w) {
    if (++w.j < w.n) return;
    w.j = 0;
    if (++w.hk < p.Hk) return;
    w.hk = 0;
    while (++w.b < p.B) {
      w.len = same(seq_len(w.b));
      w.n = tiles_of(w.len);
      if (w.n > 0) return;
    }
  };

  // ---- loads (warp-wide), as in the attention: a piece is one page's share of a tile
  const uint32_t ring = sbase + (uint32_t)(warp * L::kWarpBytes);
  const uint32_t sring = sbase + L::kScale + (uint32_t)(warp * L::kStages * L::kScaleBytes);
  const int box = p.page_size < KT ? p.page_size : KT;     // keys of a piece
  const int pieces = KT / box;                             // 1, 2 or 4
  const int nowhere = p.num_pages * p.Hk;                  // a coordinate past the cache: reads as zeros
  int issued = 0;
  auto page_at = [&](int b, int key, int len) -> int {
    return b < p.B && key < len ? p.table[(int64_t)b * p.max_pages + (key >> p.ps_log2)] : -1;
  };
  auto page_of = [&](const At& w) -> int { return page_at(w.b, w.j * KT + (lane & (KT / 16 - 1)) * box, w.len); };
  At wi = w0;
  int pages = page_of(wi);
  auto issue_next = [&]() {
    const At w = wi;
    const int pg = pages;
    advance(wi);
    pages = page_of(wi);
    const int s = issued % L::kStages;
    ++issued;
    mbar_arrive_expect_tx_w(bar(s), L::kTxBytes);
#pragma unroll 1
    for (int i = 0; i < pieces; ++i) {
      const int page = __shfl_sync(0xFFFFFFFFu, pg, i);
      const int z = page >= 0 && page < p.num_pages ? page * p.Hk + w.hk : nowhere;
      const int y = (w.j * KT + i * box) & (p.page_size - 1);
      const uint32_t dst = ring + (uint32_t)(s * L::kStageBytes + i * box * L::kRowBytes);
#pragma unroll
      for (int a = 0; a < L::kAtoms; ++a) tma_load_3d_w(dst + a * L::kAtomBytes, &tk, bar(s), 64 * a, y, z);
      if constexpr (E4M3) tma_load_2d_w(sring + (uint32_t)(s * L::kScaleBytes + i * 128), &tks, bar(s), y, z);
    }
  };
#pragma unroll 1
  for (int s = 0; s < L::kStages && s < todo; ++s) {
    if (p.stall != 0u && s >= 1) break;   // test of the timeout path: tile 1 never comes
    issue_next();
  }

  // ---- the tiles of the range
  const int g = lane >> 2, t4 = lane & 3;
  uint32_t qf[kSteps][4];
  float qs[2], lse2[2], slope2[2];
  // query row g (hh = 0) and g + 8 of this lane
  auto load_rows = [&](const At& w) {
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      const int r = g + 8 * hh;
      const bool live = r < p.R;
      const int i = live ? r / p.G : 0, h = w.hk * p.G + (live ? r % p.G : 0);
      const uint16_t* qp = p.q + ((int64_t)w.b * p.Nq + i) * p.q_tok + h * p.d;
      const float lse = live ? wp.rows_lse[((int64_t)w.b * p.Hq + h) * p.Nq + i] : INFINITY;
      // (a row that sees nothing has -inf and gives nothing)
      lse2[hh] = lse == -INFINITY ? INFINITY : lse * 1.4426950408889634f;
      slope2[hh] = p.score.slopes != nullptr ? p.score.slopes[h] * 1.4426950408889634f : 0.f;
      qs[hh] = 1.f;
#pragma unroll
      for (int c8 = 0; c8 < D / 32; ++c8) {
        // 8 dims: of the K steps 2 c8 and 2 c8 + 1 (e4m3: half of 16 dims of four steps, the same two)
        const int c = E4M3 ? 64 * (c8 >> 1) + 16 * t4 + 8 * (c8 & 1) : 32 * c8 + 8 * t4;
        const uint4 v = live && c < p.d ? *reinterpret_cast<const uint4*>(qp + c) : make_uint4(0u, 0u, 0u, 0u);
        qf[2 * c8][hh] = v.x;
        qf[2 * c8][2 + hh] = v.y;
        qf[2 * c8 + 1][hh] = v.z;
        qf[2 * c8 + 1][2 + hh] = v.w;
      }
    }
    if constexpr (E4M3 && !F16) {
      // bf16 -> fp16 by a power of two per row, as in the attention
      float top[2] = {0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 a = unpack2<false>(qf[ks][i]);
          top[i & 1] = fmaxf(top[i & 1], fmaxf(fabsf(a.x), fabsf(a.y)));
        }
      float inv[2];
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        top[hh] = fmaxf(top[hh], __shfl_xor_sync(0xFFFFFFFFu, top[hh], 1));
        top[hh] = fmaxf(top[hh], __shfl_xor_sync(0xFFFFFFFFu, top[hh], 2));
        int k = (int)(__float_as_uint(top[hh]) >> 23) - 127 - 7;
        k = k < -100 ? -100 : (k > 112 ? 112 : k);
        inv[hh] = __uint_as_float((uint32_t)(127 - k) << 23);
        qs[hh] = __uint_as_float((uint32_t)(127 + k) << 23);
      }
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 a = unpack2<false>(qf[ks][i]);
          qf[ks][i] = pack_f16x2(a.x * inv[i & 1], a.y * inv[i & 1]);
        }
    }
  };
  // the keys of a tile whose sums end in this lane (two neighbours with 64 keys)
  const int key0 = NT == 4 ? 8 * (g >> 1) + 2 * t4 + (g & 1) : 8 * g + 2 * t4;
  constexpr int kMine = NT / 4;
  At w = w0;
  bool fresh = true, ok = true;   // fresh: the next tile is the first of a (sequence, head) for this warp
#pragma unroll 1
  for (int u = 0; u < todo; ++u) {
    // where this lane's sums go, and what they are added to
    int64_t place[kMine];
    float old[kMine];
    {
      const int key = w.j * KT + key0;
      const int page = page_at(w.b, key, w.len);
      const int64_t at = ((int64_t)page * p.Hk + w.hk) * p.page_size + (key & (p.page_size - 1));
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        place[i] = page >= 0 && page < p.num_pages && key + i < w.len ? at + i : -1;
        old[i] = wp.past != nullptr && place[i] >= 0 && key + i < w.len - p.Nq ? wp.past[place[i]] : 0.f;
      }
    }
    if (fresh) load_rows(w);
    fresh = false;
    const int s = u % L::kStages;
    ok = bar_wait_warp(bar(s), (uint32_t)(u / L::kStages) & 1u, ctl, 211);
    if (!ok) break;
    // the tile as second operands: key 8 n + g, K step ks
    uint32_t kf[NT][kSteps][2];
    float2 ks2[NT];   // e4m3: the scales of keys 8 n + 2 t4 and the next
    const uint32_t sk = ring + (uint32_t)(s * L::kStageBytes);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if constexpr (!E4M3) {
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk) {
          const uint4 v = *reinterpret_cast<const uint4*>(
              smem + (sk - sbase) + (kk >> 1) * L::kAtomBytes + swz<L::kRowBytes>(8 * n + g, 4 * (kk & 1) + t4));
          kf[n][2 * kk][0] = v.x;
          kf[n][2 * kk][1] = v.y;
          kf[n][2 * kk + 1][0] = v.z;
          kf[n][2 * kk + 1][1] = v.w;
        }
      } else {
#pragma unroll
        for (int kk = 0; kk < D / 64; ++kk) {
          const uint4 v = *reinterpret_cast<const uint4*>(smem + (sk - sbase) + swz<L::kRowBytes>(8 * n + g, 4 * kk + t4));
          const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            kf[n][4 * kk + i][0] = e4m3_to_f16(x[i] & 0xFFFFu);
            kf[n][4 * kk + i][1] = e4m3_to_f16(x[i] >> 16);
          }
        }
        const int key = 8 * n + 2 * t4;
        ks2[n] = *reinterpret_cast<const float2*>(smem + (sring - sbase) + s * L::kScaleBytes +
                                                  (box == 16 ? (key >> 4) * 128 + (key & 15) * 4 : key * 4));
      }
    }
    __syncwarp();   // every lane has read the tile: its place may be loaded again
    if (issued < todo && p.stall == 0u) issue_next();
    const int left = w.len - w.j * KT;      // keys of the sequence from this tile on
    float sum[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) sum[n][0] = sum[n][1] = 0.f;
    {
      float sc[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[n][i] = 0.f;
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks)
#pragma unroll
        for (int n = 0; n < NT; ++n) mma16<F16 || E4M3>(sc[n], qf[ks], kf[n][ks][0], kf[n][ks][1]);
      const bool masked = left - (p.Nq - 1) < KT;
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int i = (g + 8 * hh) / p.G;                         // token of the row, at place len - Nq + i
        const float far = (float)(left - p.Nq + i - 2 * t4);
        const int lim = masked ? min(left - (p.Nq - 1) + i, left) : KT;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float x = sc[n][2 * hh + c];
            if constexpr (E4M3) x *= qs[hh] * (c == 0 ? ks2[n].x : ks2[n].y);
            float t = p.score.cap ? cap_any(x, p.score) : x * p.scale_log2;
            if (p.score.slopes != nullptr) t = fmaf(-slope2[hh], fabsf(far - (float)(8 * n + c)), t);
            const float e = ex2(t - lse2[hh]);
            sum[n][c] += 8 * n + 2 * t4 + c < lim ? e : 0.f;
          }
      }
    }
    float v[2 * NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      v[2 * n] = sum[n][0];
      v[2 * n + 1] = sum[n][1];
    }
    column_sums<NT>(v, g);
#pragma unroll
    for (int i = 0; i < kMine; ++i)
      if (place[i] >= 0) wp.w[place[i]] = old[i] + v[i];
    const int hk = w.hk, b = w.b;
    advance(w);
    fresh = w.hk != hk || w.b != b;
  }
  // every load issued has landed before the warp leaves (after a timeout)
  if (!ok && lane == 0) report_aborted(ctl);
  if (!ok && lane == 0)
    for (int s = 0; s < L::kStages && s < issued; ++s)
      drain_wait(bar(s), (uint32_t)((issued - 1 - s) / L::kStages) & 1u);
}

// --------------------------------------------------------------------------
// Many newest tokens (a prompt's last ones): more query rows than the 16 of a
// product, and the products, not the keys' bytes, take the time. The key tiles are
// cut into one range for each CTA, whose warps take tiles in turn; the rows of its
// (sequence, head) are staged in shared memory, up to kQRows at a time, in the
// first operand's type, and read by every warp for every tile. (Rows read from
// global memory by each warp, 16 at a time: 4 prompts of 4096-16384 tokens, 32 rows,
// 32 / 8 heads, d = 128, e4m3: 106 us, so @@.)
// --------------------------------------------------------------------------
template <int D, bool E4M3>
struct WindowLayout {
  using W = WeightsLayout<D, E4M3>;
  // (one stage: a tile goes to registers before its products, and the next one loads
  // meanwhile)
  static constexpr int kWarps = 12, kStages = 1;
  static constexpr int kQRows = 256;
  static constexpr int kPitch = D == 128 ? 320 : 192;           // of a row: 8 lanes of neighbouring rows meet no bank twice
  static constexpr int kQ = kWarps * kStages * W::kStageBytes;
  static constexpr int kScale = kQ + kQRows * kPitch;
  static constexpr int kRow = kScale + kWarps * kStages * W::kScaleBytes;   // [kQRows] x {LSE in log2 units, factor, slope, -}
  static constexpr int kBar = kRow + kQRows * 16;
  static constexpr int kMisc = kBar + 8 * kWarps * kStages;
  static constexpr int kScan = kMisc + 16;                      // int64 [kWarps] totals, int64 start, int
  static constexpr int kSmemBytes = (kScan + 8 * kWarps + 16 + 15) & ~15;
  static_assert(kSmemBytes <= 232448, "shared memory budget");
};

template <int D, bool E4M3, bool F16>
__global__ void __launch_bounds__(32 * WindowLayout<D, E4M3>::kWarps, 1)
fa_cache_window_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tks,
                       const WeightsParams wp) {
  using W = WeightsLayout<D, E4M3>;
  using L = WindowLayout<D, E4M3>;
  constexpr int KT = W::kKT, NT = KT / 8, kWarps = L::kWarps, kThreads = 32 * kWarps, kSteps = D / 16;
  const CachedParams& p = wp.c;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  auto same = [](int v) -> int { return __shfl_sync(0xFFFFFFFFu, v, 0); };   // (known to be the same in all lanes)
  const int tid = threadIdx.x, warp = same(tid >> 5), lane = tid & 31;
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  volatile uint32_t* abort_flag = misc;
  Ctl ctl{p.err, abort_flag};
  if ((sbase & 1023u) != 0u) {   // uniform across the CTA: nothing has started yet
    if (tid == 0) {
      uint32_t dummy = 0;
      Ctl c0{p.err, &dummy};
      report_error(c0, kErrSmemAlign, 212);
    }
    return;
  }
  auto bar = [&](int s) -> uint32_t { return sbase + L::kBar + 8u * (uint32_t)(warp * L::kStages + s); };
  if (lane == 0)
    for (int s = 0; s < L::kStages; ++s) mbar_init(bar(s), 1u);
  if (tid == 0) {
    misc[0] = 0u;
    misc[2] = p.wait_us;
  }
  fence_mbar_init();
  grid_dep_wait();   // global memory is read and written only from here on

  // ---- this CTA's range of the tiles of all sequences, for each the heads one after another
  const int cap = p.max_pages << p.ps_log2;
  auto seq_len = [&](int b) -> int {
    const int n = p.lens[b];
    return n < 0 ? 0 : (n > cap ? cap : n);
  };
  auto tiles_of = [&](int len) -> int { return (len + KT - 1) / KT; };
  long long* tot = reinterpret_cast<long long*>(smem + L::kScan);
  long long* start_lo = tot + kWarps;     // tiles before the sequence that the range starts in
  int* start_b = reinterpret_cast<int*>(start_lo + 1);
  const int per = (p.B + kThreads - 1) / kThreads;
  const int b_lo = min(p.B, tid * per), b_hi = min(p.B, b_lo + per);
  long long mine = 0;
  for (int b = b_lo; b < b_hi; ++b) mine += tiles_of(seq_len(b));
  long long incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long o = __shfl_up_sync(0xFFFFFFFFu, incl, off);
    if (lane >= off) incl += o;
  }
  if (lane == 31) tot[warp] = incl;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += tot[w];
    all += tot[w];
  }
  const long long total = all * p.Hk;
  const long long t0 = total * blockIdx.x / gridDim.x;
  int left_tiles = (int)(total * (blockIdx.x + 1) / gridDim.x - t0);
  long long cum = before + incl - mine;   // tiles of the sequences before b_lo
  for (int b = b_lo; b < b_hi; ++b) {
    const long long lo = cum * p.Hk, hi = (cum += tiles_of(seq_len(b))) * p.Hk;
    if (t0 >= lo && t0 < hi) {
      *start_b = b;
      *start_lo = lo;
    }
  }
  __syncthreads();
  grid_dep_launch();
  if (left_tiles == 0) return;
  int b = same(*start_b), len = same(seq_len(b)), n_tiles = tiles_of(len);
  const long long rem = t0 - *start_lo;
  int hk = same((int)(rem / n_tiles)), j0 = same((int)(rem % n_tiles));

  const uint32_t ring = sbase + (uint32_t)(warp * L::kStages * W::kStageBytes);
  const uint32_t sring = sbase + L::kScale + (uint32_t)(warp * L::kStages * W::kScaleBytes);
  const int box = p.page_size < KT ? p.page_size : KT;     // keys of a piece (one page's share of a tile)
  const int pieces = KT / box;                             // 1, 2 or 4
  const int nowhere = p.num_pages * p.Hk;                  // a coordinate past the cache: reads as zeros
  const int g = lane >> 2, t4 = lane & 3;
  const int key0 = NT == 4 ? 8 * (g >> 1) + 2 * t4 + (g & 1) : 8 * g + 2 * t4;   // (as above)
  constexpr int kMine = NT / 4;
  float4* row_of = reinterpret_cast<float4*>(smem + L::kRow);
  int issued = 0, used = 0;
  bool ok = true;
#pragma unroll 1
  while (left_tiles > 0) {
    // a (sequence, head): its tiles j0 .. j1 - 1, a warp's every kWarps-th
    const int j1 = min(n_tiles, j0 + left_tiles);
    const int m = j1 - j0 > warp ? (j1 - j0 - warp + kWarps - 1) / kWarps : 0;
    auto page_at = [&](int key) -> int {
      return key < len ? p.table[(int64_t)b * p.max_pages + (key >> p.ps_log2)] : -1;
    };
    auto issue = [&](int k) {
      if (p.stall != 0u && issued >= 1) return;   // test of the timeout path: a warp's second tile never comes
      const int j = j0 + warp + kWarps * k, s = issued % L::kStages;
      ++issued;
      const int pg = page_at(j * KT + (lane & (KT / 16 - 1)) * box);
      mbar_arrive_expect_tx_w(bar(s), W::kTxBytes);
#pragma unroll 1
      for (int i = 0; i < pieces; ++i) {
        const int page = __shfl_sync(0xFFFFFFFFu, pg, i);
        const int z = page >= 0 && page < p.num_pages ? page * p.Hk + hk : nowhere;
        const int y = (j * KT + i * box) & (p.page_size - 1);
        const uint32_t dst = ring + (uint32_t)(s * W::kStageBytes + i * box * W::kRowBytes);
#pragma unroll
        for (int a = 0; a < W::kAtoms; ++a) tma_load_3d_w(dst + a * W::kAtomBytes, &tk, bar(s), 64 * a, y, z);
        if constexpr (E4M3) tma_load_2d_w(sring + (uint32_t)(s * W::kScaleBytes + i * 128), &tks, bar(s), y, z);
      }
    };
#pragma unroll 1
    for (int r0 = 0; r0 < p.R; r0 += L::kQRows) {
      const int rows = min(L::kQRows, p.R - r0), rts = (rows + kRows - 1) / kRows;
      for (int k = 0; k < L::kStages && k < m && ok; ++k) issue(k);
      __syncthreads();   // (the rows before have been read)
      {
        // rows of D / 8 lanes, 16 bytes each
        constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;
        const int part = lane % kLanes;
        for (int r = warp * kAtOnce + lane / kLanes; r < rts * kRows; r += kWarps * kAtOnce) {
          const int row = r0 + r, i = row / p.G, h = hk * p.G + row % p.G;
          const bool live = row < p.R;
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (live && 8 * part < p.d)
            v = *reinterpret_cast<const uint4*>(p.q + ((int64_t)b * p.Nq + i) * p.q_tok + h * p.d + 8 * part);
          float factor = 1.f;
          if constexpr (E4M3 && !F16) {
            // bf16 -> fp16 by a power of two per row, as in the attention
            uint32_t x[4] = {v.x, v.y, v.z, v.w};
            float top = 0.f;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const float2 a = unpack2<false>(x[c]);
              top = fmaxf(top, fmaxf(fabsf(a.x), fabsf(a.y)));
            }
#pragma unroll
            for (int off = kLanes / 2; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, off));
            int e = (int)(__float_as_uint(top) >> 23) - 127 - 7;
            e = e < -100 ? -100 : (e > 112 ? 112 : e);
            const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
            factor = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const float2 a = unpack2<false>(x[c]);
              x[c] = pack_f16x2(a.x * inv, a.y * inv);
            }
            v = make_uint4(x[0], x[1], x[2], x[3]);
          }
          *reinterpret_cast<uint4*>(smem + L::kQ + r * L::kPitch + 16 * part) = v;
          if (part == 0) {
            // (a row that sees nothing has -inf and gives nothing)
            const float lse = live ? wp.rows_lse[((int64_t)b * p.Hq + h) * p.Nq + i] : INFINITY;
            row_of[r] = make_float4(lse == -INFINITY ? INFINITY : lse * 1.4426950408889634f, factor,
                                    live && p.score.slopes != nullptr ? p.score.slopes[h] * 1.4426950408889634f : 0.f, 0.f);
          }
        }
      }
      __syncthreads();
#pragma unroll 1
      for (int k = 0; k < m && ok; ++k) {
        const int j = j0 + warp + kWarps * k;
        // where this lane's sums go, and what they are added to
        int64_t place[kMine];
        float old[kMine];
        {
          const int key = j * KT + key0;
          const int page = page_at(key);
          const int64_t at = ((int64_t)page * p.Hk + hk) * p.page_size + (key & (p.page_size - 1));
#pragma unroll
          for (int i = 0; i < kMine; ++i) {
            place[i] = page >= 0 && page < p.num_pages && key + i < len ? at + i : -1;
            old[i] = 0.f;
            if (place[i] >= 0) {
              if (r0 > 0) old[i] = wp.w[place[i]];   // (this lane's own, of the rows before)
              else if (wp.past != nullptr && key + i < len - p.Nq) old[i] = wp.past[place[i]];
            }
          }
        }
        const int s = used % L::kStages;
        ok = bar_wait_warp(bar(s), (uint32_t)(used / L::kStages) & 1u, ctl, 213);
        if (!ok) break;
        ++used;
        uint32_t kf[NT][kSteps][2];
        float2 ks2[NT];
        const uint8_t* sk = smem + (ring - sbase) + s * W::kStageBytes;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if constexpr (!E4M3) {
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk) {
              const uint4 v = *reinterpret_cast<const uint4*>(sk + (kk >> 1) * W::kAtomBytes +
                                                              swz<W::kRowBytes>(8 * n + g, 4 * (kk & 1) + t4));
              kf[n][2 * kk][0] = v.x;
              kf[n][2 * kk][1] = v.y;
              kf[n][2 * kk + 1][0] = v.z;
              kf[n][2 * kk + 1][1] = v.w;
            }
          } else {
#pragma unroll
            for (int kk = 0; kk < D / 64; ++kk) {
              const uint4 v = *reinterpret_cast<const uint4*>(sk + swz<W::kRowBytes>(8 * n + g, 4 * kk + t4));
              const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                kf[n][4 * kk + i][0] = e4m3_to_f16(x[i] & 0xFFFFu);
                kf[n][4 * kk + i][1] = e4m3_to_f16(x[i] >> 16);
              }
            }
            const int key = 8 * n + 2 * t4;
            ks2[n] = *reinterpret_cast<const float2*>(smem + (sring - sbase) + s * W::kScaleBytes +
                                                      (box == 16 ? (key >> 4) * 128 + (key & 15) * 4 : key * 4));
          }
        }
        __syncwarp();   // every lane has read the tile: its place may be loaded again
        if (k + L::kStages < m) issue(k + L::kStages);
        const int left = len - j * KT;      // keys of the sequence from this tile on
        const bool masked = left - (p.Nq - 1) < KT;
        float sum[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) sum[n][0] = sum[n][1] = 0.f;
#pragma unroll 2
        for (int rt = 0; rt < rts; ++rt) {
          float sc[NT][4];
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) sc[n][i] = 0.f;
          const uint8_t* qr = smem + L::kQ + (rt * kRows + g) * L::kPitch;
#pragma unroll
          for (int c8 = 0; c8 < D / 32; ++c8) {
            const int c = E4M3 ? 64 * (c8 >> 1) + 16 * t4 + 8 * (c8 & 1) : 32 * c8 + 8 * t4;   // (as in load_rows)
            const uint4 v0 = *reinterpret_cast<const uint4*>(qr + 2 * c);
            const uint4 v1 = *reinterpret_cast<const uint4*>(qr + 8 * L::kPitch + 2 * c);
            const uint32_t a0[4] = {v0.x, v1.x, v0.y, v1.y}, a1[4] = {v0.z, v1.z, v0.w, v1.w};
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16<F16 || E4M3>(sc[n], a0, kf[n][2 * c8][0], kf[n][2 * c8][1]);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16<F16 || E4M3>(sc[n], a1, kf[n][2 * c8 + 1][0], kf[n][2 * c8 + 1][1]);
          }
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const int r = rt * kRows + g + 8 * hh;
            const float4 ro = row_of[r];
            const int i = (r0 + r) / p.G;                             // token of the row, at place len - Nq + i
            const float far = (float)(left - p.Nq + i - 2 * t4);
            const int lim = masked ? min(left - (p.Nq - 1) + i, left) : KT;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                float x = sc[n][2 * hh + c];
                if constexpr (E4M3) x *= ro.y * (c == 0 ? ks2[n].x : ks2[n].y);
                float u = p.score.cap ? cap_any(x, p.score) : x * p.scale_log2;
                if (p.score.slopes != nullptr) u = fmaf(-ro.z, fabsf(far - (float)(8 * n + c)), u);
                const float e = ex2(u - ro.x);
                sum[n][c] += 8 * n + 2 * t4 + c < lim ? e : 0.f;
              }
          }
        }
        float v[2 * NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          v[2 * n] = sum[n][0];
          v[2 * n + 1] = sum[n][1];
        }
        column_sums<NT>(v, g);
#pragma unroll
        for (int i = 0; i < kMine; ++i)
          if (place[i] >= 0) wp.w[place[i]] = old[i] + v[i];
      }
    }
    left_tiles -= j1 - j0;
    j0 = 0;
    if (left_tiles > 0 && ++hk == p.Hk) {
      hk = 0;
      do {
        len = same(seq_len(++b));
        n_tiles = tiles_of(len);
      } while (n_tiles == 0);
    }
  }
  // every load issued has landed before the warp leaves (after a timeout)
  if (!ok && lane == 0) report_aborted(ctl);
  if (!ok && lane == 0)
    for (int s = 0; s < L::kStages && s < issued; ++s)
      drain_wait(bar(s), (uint32_t)((issued - 1 - s) / L::kStages) & 1u);
}

template <int D, bool E4M3, bool F16>
cudaError_t launch_weights(const CUtensorMap& tk, const CUtensorMap& tks, const WeightsParams& p, cudaStream_t s) {
  using L = WeightsLayout<D, E4M3>;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static PerDeviceOnce smem_set;
  e = once_per_device(smem_set, dev, [] {
    const cudaError_t e1 = cudaFuncSetAttribute(fa_cache_weights_kernel<D, E4M3, F16>,
                                                cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmemBytes);
    return e1 != cudaSuccess ? e1
                             : cudaFuncSetAttribute(fa_cache_window_kernel<D, E4M3, F16>,
                                                    cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                    WindowLayout<D, E4M3>::kSmemBytes);
  });
  if (e != cudaSuccess) return e;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  // one CTA per SM, fewer when even full sequences have fewer tiles
  const double most = (double)p.c.B * p.c.Hk * (((double)p.c.max_pages * p.c.page_size + L::kKT - 1) / L::kKT);
  const int ctas = most < sms ? (most < 1.0 ? 1 : (int)most) : sms;
  if (p.c.RT > 1)
    return launch_pdl(true, fa_cache_window_kernel<D, E4M3, F16>, dim3((unsigned)ctas),
                      dim3(32 * WindowLayout<D, E4M3>::kWarps), WindowLayout<D, E4M3>::kSmemBytes, s, tk, tks, p);
  return launch_pdl(true, fa_cache_weights_kernel<D, E4M3, F16>, dim3((unsigned)ctas), dim3(32 * L::kWarps), L::kSmemBytes, s,
                    tk, tks, p);
}

}  // namespace

}  // namespace fa

using namespace fa;

extern "C" {

fa_status flash_attn_cached_weights(const void* Q, int64_t q_token_stride, const void* k_cache, const float* k_scale,
                                    const int32_t* block_table, const int32_t* seq_lens, const float* LSE,
                                    const float* past, float* weights, int B, int Nq, int Hq, int Hk, int d,
                                    int num_pages, int page_size, int max_pages, float scale, int cache_type,
                                    const fa_scores* scores, const fa_options* options, void* stream) {
  const bool e4m3 = cache_type == FA_CACHE_E4M3;
  bool f16 = false;
  WeightsParams p{};
  fa_status st = check_cached_call(Q, q_token_stride, k_cache, k_scale, block_table, seq_lens, B, Nq, Hq, Hk, d, num_pages,
                                   page_size, max_pages, scale, cache_type, scores, options, &f16, &p.c);
  if (st != FA_OK) return st;
  if (LSE == nullptr || weights == nullptr || !aligned(LSE, 4) || !aligned(weights, 8) || !aligned(past, 8))
    return FA_ERR_INVALID_ARG;
  const int se = internal_device_error_word(&p.c.err);
  if (se != FA_OK) return static_cast<fa_status>(se);
  p.rows_lse = LSE;
  p.past = past;
  p.w = weights;
  const int D = d <= 64 ? 64 : 128;
  const uint32_t keys = 4096u / (uint32_t)D;
  CUtensorMap tk, tks;
  if (!cached_maps(&tk, &tks, k_cache, k_scale, e4m3, f16, Hk, d, num_pages, page_size, keys)) return FA_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaErrorInvalidValue;
#define FA_WEIGHTS_CASE(DD, EE, FF) \
  if (D == DD && e4m3 == EE && f16 == FF) e = launch_weights<DD, EE, FF>(tk, tks, p, s);
  FA_WEIGHTS_CASE(64, false, false)
  FA_WEIGHTS_CASE(64, false, true)
  FA_WEIGHTS_CASE(64, true, false)
  FA_WEIGHTS_CASE(64, true, true)
  FA_WEIGHTS_CASE(128, false, false)
  FA_WEIGHTS_CASE(128, false, true)
  FA_WEIGHTS_CASE(128, true, false)
  FA_WEIGHTS_CASE(128, true, true)
#undef FA_WEIGHTS_CASE
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
