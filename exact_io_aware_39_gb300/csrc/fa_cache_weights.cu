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
// (64 sequences of 144891 tokens in all, 32 / 8 heads, d = 128, bf16, capped scores:
// 57 us, 5.3 TB/s of 6.8.)
//
// The 16 bytes a lane reads of a key are 8 neighbouring dims (16 in e4m3), which
// it spreads over two (four) K steps of the product; the queries are read in the
// same order, so that a lane reads them by 16 bytes as well.
#include "fa_cached.cuh"
#include "fa_packed.cuh"

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

// Adds the weights of a row against a tile to its keys' sums: x are its raw products
// with keys 8 n + 2 t4 + c, mul (times `factor`, e4m3) brings them to scores (to log2
// units where there is no cap), far is the row's place less the lane's first key;
// keys from column lim on are not seen (masked).
template <int NT, bool E4M3>
__device__ __forceinline__ void add_weights(float (&sum)[NT][2], const float (&x)[NT][2], const float2 (&mul)[E4M3 ? NT : 1],
                                            float factor, float lse2, float slope2, float far, bool masked, int lim,
                                            int first, const ScoreParams& sp) {
  float u[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    u[n][0] = x[n][0] * (E4M3 ? factor * mul[E4M3 ? n : 0].x : mul[0].x);
    u[n][1] = x[n][1] * (E4M3 ? factor * mul[E4M3 ? n : 0].y : mul[0].x);
  }
  if (sp.cap) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) u[n][c] = cap_any(u[n][c], sp);
  }
  if (sp.slopes != nullptr) {   // (keys past the row's place are masked)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) u[n][c] = fmaf(-slope2, far - (float)(8 * n + c), u[n][c]);
  }
  if (masked) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c)
        if (8 * n + first + c >= lim) u[n][c] = -INFINITY;
  }
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int c = 0; c < 2; ++c) sum[n][c] += ex2(u[n][c] - lse2);
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
  // query row g (hh = 0) and g + 8 of this lane. Rows behind the last are copies of it, which sees every key,
  // with an LSE of inf: they give nothing, and a NaN only where the last row does (zeros would give one with
  // an infinite element).
  auto load_rows = [&](const At& w) {
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      const int r = g + 8 * hh;
      const bool live = r < p.R;
      const int row = live ? r : p.R - 1, i = row / p.G, h = w.hk * p.G + row % p.G;
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
        const uint4 v = c < p.d ? *reinterpret_cast<const uint4*>(qp + c) : make_uint4(0u, 0u, 0u, 0u);
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
    const float unit = p.score.cap ? 1.f : p.scale_log2;
    float2 mul[E4M3 ? NT : 1];   // of products with keys 8 n + 2 t4 and the next (e4m3: with their scales)
    if constexpr (!E4M3) mul[0] = make_float2(unit, unit);
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
        const float2 ks = *reinterpret_cast<const float2*>(smem + (sring - sbase) + s * L::kScaleBytes +
                                                           (box == 16 ? (key >> 4) * 128 + (key & 15) * 4 : key * 4));
        mul[n] = make_float2(ks.x * unit, ks.y * unit);
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
        if (hh == 1 && p.R <= 8) break;
        const int i = (g + 8 * hh) / p.G;                         // token of the row, at place len - Nq + i
        float x[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          x[n][0] = sc[n][2 * hh];
          x[n][1] = sc[n][2 * hh + 1];
        }
        add_weights<NT, E4M3>(sum, x, mul, qs[hh], lse2[hh], slope2[hh], (float)(left - p.Nq + i - 2 * t4), masked,
                              min(left - (p.Nq - 1) + i, left), 2 * t4, p.score);
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
// Many newest tokens (a prompt's last ones): more query rows than the 16 of an
// mma.sync product, and the products, not the keys' bytes, take the time: tcgen05,
// S^T = K Q^T in TMEM, 128 keys by up to 128 rows. A thread is a key and adds its
// weights up over the columns, so the rows' sums need no exchange at all.
//
// The key tiles of all (sequence, head) pairs are cut into one range for each CTA.
// Roles: a producer warp loads tiles by TMA into a ring; with e4m3 four warps convert
// them (exactly) to fp16 operand tiles; an MMA warp issues each product into one of
// four TMEM buffers, which four warpgroups read in turn. The rows of the range's
// (sequence, head) are staged in shared memory by the groups, kQRows at a time,
// in the first operand's type; keys are read again for every kQRows rows (those behind
// the block's last token too, though none of it sees them: 2 prompts of 2048 tokens, all
// of them queries, 32 / 8 heads, d = 128, e4m3, 357 us). The roles
// that read the rows meet at two named barriers for each such block; one whose wait
// failed goes on to meet them there, without working.
// (4 prompts of 4096-16384 tokens, 32 of them new, 32 / 8 heads, d = 128, e4m3, inputs
// out of the cache: 30 us, 37 with two warpgroups; with mma.sync and rows read from global
// memory 106, from shared memory 55. 43 MB of keys take 6: a CTA has about 17 tiles of
// 0.45 us, by the conversion, and spends 4 us on each block of rows and 3 on the lengths.
// Among other calls 23 us, in bf16 19; capped 57 and 40, lowered with distance 30: the
// general loop forms both tanhs of every score.)
// --------------------------------------------------------------------------
template <int D, bool E4M3>
struct WindowLayout {
  static constexpr int kKeys = kTile, kQRows = 128;
  static constexpr int kTileBytes = kKeys * D * 2;              // an operand tile, 64-column atoms 16 KB apart
  static constexpr int kRawBytes = E4M3 ? kKeys * D : kTileBytes;
  static constexpr int kRawRow = E4M3 ? D : 128;                // bytes of a row as the TMA writes it
  static constexpr int kStages = 4;
  static constexpr int kGroups = 4, kSums = 4 * kGroups;        // warpgroups that read S, and their warps
  static constexpr int kConverters = E4M3 ? 4 : 0;
  static constexpr int kProducer = kSums + kConverters, kMma = kProducer + 1, kThreads = 32 * (kMma + 1);
  static constexpr int kConv = kStages * kRawBytes;             // [2] tiles (e4m3)
  static constexpr int kQ = kConv + (E4M3 ? 2 * kTileBytes : 0);
  static constexpr int kRow = kQ + kQRows * D * 2;              // [kQRows] each: factor, -LSE in log2 units, slope, token
  static constexpr int kBar = kRow + kQRows * 16;
  static constexpr int bFull = 0;                               // [kStages]
  static constexpr int bEmpty = bFull + kStages;                // [kStages]: converted, or read by the product
  static constexpr int bConvFull = bEmpty + kStages;            // [2], 4 arrivals
  static constexpr int bConvEmpty = bConvFull + 2;              // [2]
  static constexpr int bSFull = bConvEmpty + 2;                 // [kGroups]
  static constexpr int bSEmpty = bSFull + kGroups;              // [kGroups], 4: S has been read
  static constexpr int bDrain = bSEmpty + kGroups;
  static constexpr int kNumBars = bDrain + 1;
  static constexpr int kMisc = (kBar + 8 * kNumBars + 15) & ~15;   // tmem slot, abort flag, -, wait limit
  static constexpr int kExp = kMisc + 16;                       // int [2]{largest, smallest exponent of a row}, by turns
  static constexpr int kScan = kExp + 16;                       // int64 [kMma + 1] totals, int64 start, int
  static constexpr int kSmemBytes = (kScan + 8 * (kMma + 1) + 16 + 15) & ~15;
  static_assert(kSmemBytes <= 232448, "shared memory budget");
};

template <int D, bool E4M3, bool F16>
__global__ void __launch_bounds__(WindowLayout<D, E4M3>::kThreads, 1)
fa_cache_window_kernel(const __grid_constant__ CUtensorMap tk, const WeightsParams wp, const float* __restrict__ k_scale) {
  using L = WindowLayout<D, E4M3>;
  constexpr bool PF16 = E4M3 || F16;     // the operands' type
  constexpr uint32_t kRowsBar = 1u, kReadyBar = 2u;   // named: the rows may be replaced; they are staged
  const CachedParams& p = wp.c;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  auto same = [](int v) -> int { return __shfl_sync(0xFFFFFFFFu, v, 0); };   // (known to be the same in all lanes)
  const int tid = threadIdx.x, warp = same(tid >> 5), lane = tid & 31;
  auto bar = [&](int i) -> uint32_t { return sbase + L::kBar + 8u * (uint32_t)i; };
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  volatile uint32_t* abort_flag = misc + 1;
  Ctl ctl{p.err, abort_flag};
  if ((sbase & 1023u) != 0u) {   // uniform across the CTA: nothing has started yet
    if (tid == 0) {
      uint32_t dummy = 0;
      Ctl c0{p.err, &dummy};
      report_error(c0, kErrSmemAlign, 212);
    }
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < L::kNumBars; ++i)
      mbar_init(bar(i), (i >= L::bSEmpty && i < L::bSEmpty + L::kGroups) || (i >= L::bConvFull && i < L::bConvFull + 2) ||
                                (E4M3 && i >= L::bEmpty && i < L::bEmpty + L::kStages)
                            ? 4u : 1u);
    abort_flag[0] = 0u;
    abort_flag[2] = p.wait_us;   // the wait limit, read by the slow path of every wait
    int* exps = reinterpret_cast<int*>(smem + L::kExp);
    exps[0] = exps[2] = -1000;
    exps[1] = exps[3] = 1000;
    fence_mbar_init();
  }
  if (warp == L::kMma) {
    tmem_alloc(smem_u32(misc), 128 * L::kGroups);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();   // the barriers are initialised and TMEM allocated
  tc_fence_after();
  const uint32_t tmem = misc[0];
  grid_dep_wait();   // global memory is read and written only from here on

  // ---- this CTA's range of the tiles of all sequences, for each the heads one after another
  const int cap = p.max_pages << p.ps_log2;
  auto seq_len = [&](int b) -> int {
    const int n = p.lens[b];
    return n < 0 ? 0 : (n > cap ? cap : n);
  };
  auto tiles_of = [&](int len) -> int { return (len + L::kKeys - 1) / L::kKeys; };
  constexpr int kWarps = L::kMma + 1;
  long long* tot = reinterpret_cast<long long*>(smem + L::kScan);
  long long* start_lo = tot + kWarps;     // tiles before the sequence that the range starts in
  int* start_b = reinterpret_cast<int*>(start_lo + 1);
  const int per = (p.B + L::kThreads - 1) / L::kThreads;
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
  // a role's walk over the range: blocks of rows of (sequence, head)s, tiles j0 .. j1 - 1
  int b = 0, len = 0, n_tiles = 1, hk = 0, j0 = 0, j1 = 0, g = 0;   // g: tiles so far
  if (left_tiles > 0) {
    b = same(*start_b);
    len = same(seq_len(b));
    n_tiles = tiles_of(len);
    const long long rem = t0 - *start_lo;
    hk = same((int)(rem / n_tiles));
    j0 = same((int)(rem % n_tiles));
  }
  auto walk = [&](auto&& block) {
    while (left_tiles > 0) {
      j1 = min(n_tiles, j0 + left_tiles);
      for (int r0 = 0; r0 < p.R; r0 += L::kQRows) block(r0);
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
  };
  auto page_at = [&](int key) -> int {
    const int page = key < len ? p.table[(int64_t)b * p.max_pages + (key >> p.ps_log2)] : -1;
    return page < p.num_pages ? page : -1;
  };
  bool ok = true;
  if (warp == L::kProducer) {
    // ------------------------------------------------------------ loads (a piece is one page's share of a tile)
    if (lane == 0) tma_prefetch_map(&tk);
    const int box = p.page_size < L::kKeys ? p.page_size : L::kKeys;
    const int pieces = L::kKeys / box;                       // 1 to 8
    const int nowhere = p.num_pages * p.Hk;                  // a coordinate past the cache: reads as zeros
    const int batch = 32 / pieces;                           // tiles whose pages the lanes hold
    int issued = 0;
    walk([&](int) {
      // the pages of the next batch are on their way while this one's tiles are loaded
      int pages = 0, next = page_at((j0 + lane / pieces) * L::kKeys + (lane % pieces) * box);
      for (int j = j0; j < j1 && ok; ++j, ++g) {
        if (p.stall != 0u && g >= 1) { ok = false; break; }   // test of the timeout path: tile 1 never comes
        const int s = g % L::kStages, at = (j - j0) % batch;
        if (at == 0) {
          pages = next;
          next = page_at((j + batch + lane / pieces) * L::kKeys + (lane % pieces) * box);
        }
        if (g >= L::kStages && !(ok = bar_wait_warp(bar(L::bEmpty + s), (uint32_t)(g / L::kStages - 1) & 1u, ctl, 213))) break;
        mbar_arrive_expect_tx_w(bar(L::bFull + s), L::kRawBytes);
        ++issued;
#pragma unroll 1
        for (int i = 0; i < pieces; ++i) {
          const int page = __shfl_sync(0xFFFFFFFFu, pages, at * pieces + i);
          const int z = page >= 0 ? page * p.Hk + hk : nowhere;
          const int y = (j * L::kKeys + i * box) & (p.page_size - 1);
          const uint32_t dst = sbase + (uint32_t)(s * L::kRawBytes + i * box * L::kRawRow);
#pragma unroll
          for (int a = 0; a < (E4M3 ? 1 : D / 64); ++a) tma_load_3d_w(dst + a * 16384, &tk, bar(L::bFull + s), 64 * a, y, z);
        }
      }
    });
    // every load issued has landed before the CTA exits
    if (lane == 0)
      for (int s = 0; s < L::kStages && s < issued; ++s)
        drain_wait(bar(L::bFull + s), (uint32_t)((issued - 1 - s) / L::kStages) & 1u);
  } else if (warp == L::kMma) {
    // ------------------------------------------------------------ products (warp-wide, one elected lane issues)
    const uint32_t dQ = desc_lo(desc_kmajor(sbase + L::kQ, 0));
    walk([&](int r0) {
      named_bar_sync(kReadyBar, 32u * (L::kSums + 1));
      tc_fence_after();
      const int N = (min(L::kQRows, p.R - r0) + 15) & ~15;
      const uint32_t id = idesc_16<PF16>(128, N, false, false);
      for (int j = j0; j < j1 && ok; ++j, ++g) {
        const int s = E4M3 ? g & 1 : g % L::kStages, buf = g % L::kGroups;
        const uint32_t n = (uint32_t)(g / (E4M3 ? 2 : L::kStages));
        if (!(ok = bar_wait_warp(bar((E4M3 ? L::bConvFull : L::bFull) + s), n & 1u, ctl, 214))) break;
        if (g >= L::kGroups && !(ok = bar_wait_warp(bar(L::bSEmpty + buf), (uint32_t)(g / L::kGroups - 1) & 1u, ctl, 215)))
          break;
        tc_fence_after();
        const uint32_t dK = desc_lo(desc_kmajor(sbase + (E4M3 ? L::kConv : 0) + s * L::kTileBytes, 0));
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          mma_ss_lo(tmem + 128u * (uint32_t)buf, dK + (uint32_t)kmajor_step(ks), dQ + (uint32_t)kmajor_step(ks), id,
                    ks > 0 ? 1u : 0u);
        mma_commit_w(bar(L::bSFull + buf));
        mma_commit_w(bar((E4M3 ? L::bConvEmpty : L::bEmpty) + s));
      }
    });
    // every MMA issued has completed before TMEM is freed
    mma_commit_w(bar(L::bDrain));
    drain_wait(bar(L::bDrain), 0);
  } else if (E4M3 && warp >= L::kSums && warp < L::kSums + L::kConverters) {
    // ------------------------------------------------------------ e4m3 -> fp16 (thread = key)
    const int r = tid - 32 * L::kSums;
    walk([&](int) {
      for (int j = j0; j < j1 && ok; ++j, ++g) {
        const int s = g % L::kStages, c = g & 1;
        if (!(ok = bar_wait_warp(bar(L::bFull + s), (uint32_t)(g / L::kStages) & 1u, ctl, 216))) break;
        if (g >= 2 && !(ok = bar_wait_warp(bar(L::bConvEmpty + c), (uint32_t)(g / 2 - 1) & 1u, ctl, 217))) break;
        const uint8_t* raw = smem + s * L::kRawBytes;
        uint8_t* out = smem + L::kConv + c * L::kTileBytes;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const uint4 v = *reinterpret_cast<const uint4*>(raw + swz<L::kRawRow>(r, i));
          *reinterpret_cast<uint4*>(out + tile_chunk(r, 2 * i)) =
              make_uint4(e4m3_to_f16(v.x & 0xFFFFu), e4m3_to_f16(v.x >> 16), e4m3_to_f16(v.y & 0xFFFFu), e4m3_to_f16(v.y >> 16));
          *reinterpret_cast<uint4*>(out + tile_chunk(r, 2 * i + 1)) =
              make_uint4(e4m3_to_f16(v.z & 0xFFFFu), e4m3_to_f16(v.z >> 16), e4m3_to_f16(v.w & 0xFFFFu), e4m3_to_f16(v.w >> 16));
        }
        fence_proxy_async_smem();
        mbar_arrive_warp(bar(L::bConvFull + c));
        mbar_arrive_warp(bar(L::bEmpty + s));
      }
    });
  } else if (warp < L::kSums) {
    // ------------------------------------------------------------ weights (thread = key)
    const int wg = warp >> 2, r = tid & 127;
    const uint32_t tS = tmem + 128u * (uint32_t)wg + ((uint32_t)((warp & 3) * 32) << 16);
    float* r_mul = reinterpret_cast<float*>(smem + L::kRow);
    float *r_lse = r_mul + L::kQRows, *r_slope = r_lse + L::kQRows, *r_tok = r_slope + L::kQRows;
    const float unit = p.score.cap ? 1.f : p.scale_log2;
    const bool plain = !p.score.cap && p.score.slopes == nullptr;
    int turn = 0;
    walk([&](int r0) {
      const int rows = min(L::kQRows, p.R - r0), cols = (rows + 15) & ~15;
      named_bar_sync(kRowsBar, 32u * L::kSums);   // (the rows before have been read)
      // all that the block reads from global memory is on its way before the first of it is waited for:
      // the rows' elements, D / 8 lanes a row, 16 bytes each
      constexpr int kLanes = D / 8, kStep = L::kSums * (32 / kLanes), kRowsEach = L::kQRows / kStep;
      const int part = lane % kLanes, q0 = warp * (32 / kLanes) + lane / kLanes;
      uint4 v[kRowsEach];
#pragma unroll
      for (int n = 0; n < kRowsEach; ++n) {
        const int q = q0 + n * kStep, row = r0 + q, i = row / p.G, h = hk * p.G + row % p.G;
        v[n] = make_uint4(0u, 0u, 0u, 0u);
        if (q < rows && 8 * part < p.d)
          v[n] = *reinterpret_cast<const uint4*>(p.q + ((int64_t)b * p.Nq + i) * p.q_tok + h * p.d + 8 * part);
      }
      // and where the groups' tiles' sums go and what they are added to: read one of its tiles ahead, the pages two.
      // Behind the first rows that is this CTA's own sum (past may be w).
      const int t_first = j0 + ((wg - g) & (L::kGroups - 1));
      auto page_in = [&](int j) -> int { return j < j1 ? page_at(j * L::kKeys + r) : -1; };
      int page0 = page_in(t_first), page1 = page_in(t_first + L::kGroups);
      const float* sums = r0 > 0 ? wp.w : wp.past;
      const int sums_to = sums == nullptr ? 0 : (r0 > 0 ? len : len - p.Nq);
      auto place_of = [&](int j, int page) -> int64_t {
        return ((int64_t)page * p.Hk + hk) * p.page_size + ((j * L::kKeys + r) & (p.page_size - 1));
      };
      float old0 = 0.f, ks0 = 1.f;
      if (tid < cols) {
        // (a row that sees nothing has -inf and gives nothing; the rows behind the last see no key, whose
        // elements may be infinite)
        const int row = r0 + tid, i = row / p.G, h = hk * p.G + row % p.G;
        const bool live = tid < rows;
        const float lse = live ? wp.rows_lse[((int64_t)b * p.Hq + h) * p.Nq + i] : INFINITY;
        r_lse[tid] = lse == -INFINITY ? -INFINITY : lse * -1.4426950408889634f;
        r_slope[tid] = live && p.score.slopes != nullptr ? p.score.slopes[h] * 1.4426950408889634f : 0.f;
        r_tok[tid] = live ? (float)i : -INFINITY;
      }
      // bf16 beside e4m3: to fp16 by a power of two, as in the attention (its largest element gets 2^7 to 2^8).
      // The rows share the largest one's where the smallest is within 2^6 of it (what falls below fp16's
      // smallest then is off by at most 2^-26 of the row's largest): no product by a row's own is left.
      float mul = unit;
      bool shared = true;
      if constexpr (E4M3 && !F16) {
        int* exps = reinterpret_cast<int*>(smem + L::kExp) + 2 * (turn & 1);
        int ex[kRowsEach];
#pragma unroll
        for (int n = 0; n < kRowsEach; ++n) {
          const uint32_t x[4] = {v[n].x, v[n].y, v[n].z, v[n].w};
          float top = 0.f;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float2 a = unpack2<false>(x[c]);
            top = fmaxf(top, fmaxf(fabsf(a.x), fabsf(a.y)));
          }
#pragma unroll
          for (int off = kLanes / 2; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, off));
          const int e = (int)(__float_as_uint(top) >> 23) - 127 - 7;
          ex[n] = e < -100 ? -100 : (e > 112 ? 112 : e);
          if (part == 0 && top > 0.f) {
            atomicMax(exps, ex[n]);
            atomicMin(exps + 1, ex[n]);
          }
        }
        named_bar_sync(kRowsBar, 32u * L::kSums);
        const int hi = max(exps[0], -100);   // (-1000: all rows are zeros)
        shared = hi - exps[1] <= 6;
        mul = unit * __uint_as_float((uint32_t)(127 + hi) << 23);
        ++turn;
        if (tid == 0) {   // (the next block's, which have been read: all are past the barrier above)
          int* other = reinterpret_cast<int*>(smem + L::kExp) + 2 * (turn & 1);
          other[0] = -1000;
          other[1] = 1000;
        }
#pragma unroll
        for (int n = 0; n < kRowsEach; ++n) {
          const int e = shared ? hi : ex[n], q = q0 + n * kStep;
          const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
          uint32_t x[4] = {v[n].x, v[n].y, v[n].z, v[n].w};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float2 a = unpack2<false>(x[c]);
            x[c] = pack_f16x2(a.x * inv, a.y * inv);
          }
          v[n] = make_uint4(x[0], x[1], x[2], x[3]);
          if (part == 0 && q < cols) r_mul[q] = unit * __uint_as_float((uint32_t)(127 + e) << 23);
        }
      }
#pragma unroll
      for (int n = 0; n < kRowsEach; ++n)
        if (q0 + n * kStep < cols) *reinterpret_cast<uint4*>(smem + L::kQ + tile_chunk(q0 + n * kStep, part)) = v[n];
      if (page0 >= 0) {
        const int64_t place = place_of(t_first, page0);
        if (t_first * L::kKeys + r < sums_to) old0 = sums[place];
        if constexpr (E4M3) ks0 = k_scale[place];
      }
      fence_proxy_async_smem();
      named_bar_sync(kReadyBar, 32u * (L::kSums + 1));
      for (int j = j0; j < j1; ++j, ++g) {
        if (!ok || (g & (L::kGroups - 1)) != wg) continue;
        const int key = j * L::kKeys + r, page = page0;
        const float old = old0, ks = shared ? ks0 * mul : ks0;   // (what the products are multiplied by)
        page0 = page1;
        page1 = page_in(j + 2 * L::kGroups);
        if (page0 >= 0) {
          const int64_t place = place_of(j + L::kGroups, page0);
          if (key + L::kGroups * L::kKeys < sums_to) old0 = sums[place];
          else old0 = 0.f;
          if constexpr (E4M3) ks0 = k_scale[place];
        }
        // query i is at place len - Nq + i: it sees the key from i = key - (len - Nq) on
        const float behind = (float)(len - p.Nq - key);
        const bool masked = j * L::kKeys + L::kKeys > len - p.Nq + 1;
        if (!(ok = bar_wait_warp(bar(L::bSFull + wg), (uint32_t)(g / L::kGroups) & 1u, ctl, 218))) continue;
        tc_fence_after();
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        const float2 k2 = make_float2(ks, ks);
        if (plain && shared && !masked && (rows & 15) == 0) {
          // (nothing but these in the loop: the compiler then overlaps one column's latencies with another's)
#pragma unroll 1
          for (int c = 0; c < cols; c += 16) {
            uint32_t u[16];
            tmem_ld16(tS + (uint32_t)c, u);
            float2 x[8];
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
              const float4 l4 = *reinterpret_cast<const float4*>(r_lse + c + 2 * i);
              x[i] = __ffma2_rn(make_float2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1])), k2, make_float2(l4.x, l4.y));
              x[i + 1] = __ffma2_rn(make_float2(__uint_as_float(u[2 * i + 2]), __uint_as_float(u[2 * i + 3])), k2,
                                    make_float2(l4.z, l4.w));
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[i & 1] = __fadd2_rn(sum[i & 1], make_float2(ex2(x[i].x), ex2(x[i].y)));
          }
        } else {
#pragma unroll 1
          for (int c = 0; c < cols; c += 16) {
            uint32_t u[16];
            tmem_ld16(tS + (uint32_t)c, u);
            auto pair = [&](const float* of, int i) -> float2 { return *reinterpret_cast<const float2*>(of + c + 2 * i); };
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float2 x = make_float2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]));
              if (E4M3 && !F16 && !shared) x = __fmul2_rn(x, pair(r_mul, i));
              x = __fmul2_rn(x, k2);
              if (p.score.cap) x = make_float2(cap_any(x.x, p.score), cap_any(x.y, p.score));
              const float2 s = pair(r_slope, i), far = __fadd2_rn(make_float2(behind, behind), pair(r_tok, i));
              x = __fadd2_rn(__ffma2_rn(make_float2(-s.x, -s.y), far, x), pair(r_lse, i));
              // (keys past the row's place, and rows behind the last)
              x = make_float2(far.x < 0.f ? -INFINITY : x.x, far.y < 0.f ? -INFINITY : x.y);
              sum[i & 1] = __fadd2_rn(sum[i & 1], make_float2(ex2(x.x), ex2(x.y)));
            }
          }
        }
        tc_fence_before();
        mbar_arrive_warp(bar(L::bSEmpty + wg));
        const float2 both = __fadd2_rn(sum[0], sum[1]);
        if (page >= 0) wp.w[place_of(j, page)] = old + (both.x + both.y);
      }
    });
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0) report_aborted(ctl);
  if (warp == L::kMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 128 * L::kGroups);
  }
}

template <int D, bool E4M3, bool F16>
cudaError_t launch_weights(const CUtensorMap& tk, const CUtensorMap& tks, const WeightsParams& p, const float* k_scale,
                           cudaStream_t s) {
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
  const int keys = p.c.RT > 1 ? WindowLayout<D, E4M3>::kKeys : L::kKT;
  const double most = (double)p.c.B * p.c.Hk * (((double)p.c.max_pages * p.c.page_size + keys - 1) / keys);
  const int ctas = most < sms ? (most < 1.0 ? 1 : (int)most) : sms;
  if (p.c.RT > 1)
    return launch_pdl(true, fa_cache_window_kernel<D, E4M3, F16>, dim3((unsigned)ctas),
                      dim3(WindowLayout<D, E4M3>::kThreads), WindowLayout<D, E4M3>::kSmemBytes, s, tk, p, k_scale);
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
  const int keys = p.c.RT > 1 ? kTile : 4096 / D;
  CUtensorMap tk, tks;
  if (!cached_maps(&tk, &tks, k_cache, k_scale, e4m3, f16, Hk, d, num_pages, page_size, keys)) return FA_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaErrorInvalidValue;
#define FA_WEIGHTS_CASE(DD, EE, FF) \
  if (D == DD && e4m3 == EE && f16 == FF) e = launch_weights<DD, EE, FF>(tk, tks, p, k_scale, s);
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
