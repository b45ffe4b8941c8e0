// Serving from a paged key/value cache, for sm_103a: the writer (16-bit copy
// or quantisation to e4m3 with one scale per row) and the attention of the
// newest tokens against the cache. Declarations and the contract of the calls
// are in flash_attn_cache.h.
//
// Attention of the newest tokens. Per sequence and key/value head there are
// Nq * G query rows (G = Hq / Hk; 1 to 16 as a rule) against thousands of
// keys, so the work is reading the cache: 2 d elements per key for 4 d Nq G
// operations, far under the 280 operations per byte where the tensor cores
// would bound it. The design keeps the memory system busy and little else:
//   * the unit of work is a tile of 16 to 64 keys of one (sequence, key/value
//     head, 16 query rows); all units of the call are numbered in that order and
//     cut into equal ranges, one for each warp of the grid, so that ragged
//     lengths leave no warp without work;
//   * each warp is a pipeline of its own: it loads the tiles of its range by
//     TMA into its own shared-memory ring, across sequence boundaries, so an SM
//     keeps up to 192 KB in flight (6.8 TB/s x 1 us / 152 = 45 KB are needed), and
//     no warp waits for another;
//   * the products are mma.sync m16n8k16: the 16 rows fill it, where a
//     tcgen05 product of 128 rows would be an eighth full or less, and the
//     operands come from registers (Q, P, and with e4m3 the converted K and V);
//   * calls of few, short sequences are served by a cluster per (sequence, head)
//     instead, in one launch (WHOLE, below);
//   * a warp that finishes a (sequence, head) whole writes O and the LSE; one
//     that holds a part of it writes O unnormalised with the row's reference
//     and sum, and a second kernel joins the parts (in a fixed order, so the
//     result does not change from call to call).
// Measured (the kernels, replayed from a graph), 32 query and 8 key/value heads,
// d = 128: 64 sequences of 144891 tokens in all (512-8192 each) in bf16 101 us with
// the join (5.9 TB/s of 6.8), 16 of 485214 in all (8192-65536 each) in e4m3 161 us
// (6.4 TB/s); one of 500 tokens 6.8 us. The sizes below are those of these calls
// where no other number of tokens is given.
//
// e4m3: with q8, k8, v8 the payloads and ks, vs the scales of key j,
//   S_j = ks_j (q . k8_j),  O = sum_j P_j vs_j v8_j.
// The payloads are converted exactly to fp16; Q is brought into fp16's range
// by a power of two per row. The weights w_j = P_j vs_j that go to fp16 for
// the second product are formed as 2^(s_j + log2 vs_j - m) with m the running
// maximum of s_j + log2 vs_j, so they are at most 2^8 and lose nothing to
// fp16's range however the scales differ; the row sum adds w_j / vs_j in fp32.
// A value scale of 0 (a page outside the cache reads so, and a scale tensor may
// start so) has no logarithm: it becomes the writer's smallest scale, so that its
// w_j outweighs no other, and its row of V zeros in shared memory. (Looking for
// them among the scales in registers takes 0.7 % of a call on 16 sequences of
// 381292 tokens in all, d = 128, and 3 % of one on 16000; replacing each as it is
// used took 6 % of the former, looking in shared memory ahead of the products 2.5.)
#include "flash_attn_cache.h"
#include "fa_common.cuh"
#include "fa_ptx.cuh"
#include "fa_warp.cuh"

#include <cmath>

namespace fa {

namespace {

// --------------------------------------------------------------------------
// writer
// --------------------------------------------------------------------------

struct WriteParams {
  const uint16_t* src[2];      // K, V
  int64_t tok[2], head[2];     // strides in elements
  const int64_t* slots;
  void* cache[2];
  float* scale[2];
  uint32_t rows;               // T Hk of each tensor
  uint32_t Hk;
  uint64_t magic;              // row / Hk = (row * magic) >> 37 (see write_magic)
  int d;
  int ps_log2;
  int64_t places;              // num_pages * page_size
};

// Rows from which on a thread takes two rows of a tensor instead of one. (To
// e4m3, 8 heads, d = 128: 32768 tokens 34.1 us with two rows, 35.7 with one, 37.9
// with four -- 6.0 TB/s; 4096 tokens 5.7 and 5.6; as they are, 32768 tokens
// 41.1 and 44.2 us -- 6.5 TB/s.)
constexpr uint32_t kManyRows = 65536;

// Division of a row number r < 2^27 by Hk <= 2^10: (r * m) >> 37 with
// m = ceil(2^37 / Hk) is exact while r * (m Hk - 2^37) < 2^37, and
// m Hk - 2^37 < Hk; r * m stays under 2^64.
constexpr int kMaxWriteHeads = 1024;
constexpr double kMaxWriteRows = 67108864.0;   // 2^26, and a block's rows past the end
uint64_t write_magic(int Hk) { return (((uint64_t)1 << 37) + (uint64_t)Hk - 1) / (uint64_t)Hk; }

__device__ __forceinline__ uint16_t cvt_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// A row (token, head) of K or V (blockIdx.y) is handled by LANES neighbouring
// threads of kE elements each, U rows by the same threads, their loads before
// anything waits for one; rows are numbered heads first, so that a block reads
// neighbouring tokens' heads in one piece. Bound by memory: 2 + 1 bytes per
// element to e4m3, 2 + 2 as they are.
//
// e4m3: the row's largest magnitude is taken over the 16-bit patterns (without
// their signs these order as the values do, infinities and NaN above all), two
// to a word; only a row that holds an infinity or NaN looks at single elements.
template <int LANES, int U, bool E4M3, bool F16>
__global__ void __launch_bounds__(256) kv_cache_write_kernel(const WriteParams p) {
  constexpr int kE = E4M3 ? 16 : 8;
  constexpr int kW = kE / 8;                  // 16-byte words of a lane
  constexpr uint32_t kGroups = 256 / LANES;   // rows a block takes at a time
  const int part = (int)(threadIdx.x % LANES);
  const bool is_v = blockIdx.y != 0;
  const uint16_t* const src0 = is_v ? p.src[1] : p.src[0];
  const int64_t tok = is_v ? p.tok[1] : p.tok[0], head = is_v ? p.head[1] : p.head[0];
  void* const cache = is_v ? p.cache[1] : p.cache[0];
  const uint32_t row0 = blockIdx.x * (kGroups * U) + threadIdx.x / LANES;
  const bool cols = kE * part < p.d;
  uint4 x[U][kW];
  int64_t place[U];   // row of the cache, or -1
  grid_dep_wait();
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t row = row0 + (uint32_t)u * kGroups;
    const uint32_t t = (uint32_t)(((uint64_t)row * p.magic) >> 37);
    const uint32_t h = row - t * p.Hk;
#pragma unroll
    for (int i = 0; i < kW; ++i) x[u][i] = make_uint4(0u, 0u, 0u, 0u);
    place[u] = -1;
    if (row < p.rows && cols) {
      const int64_t slot = p.slots[t];
      const uint16_t* src = src0 + (int64_t)t * tok + (int64_t)h * head + kE * part;
#pragma unroll
      for (int i = 0; i < kW; ++i) x[u][i] = *reinterpret_cast<const uint4*>(src + 8 * i);
      if (slot >= 0 && slot < p.places)
        place[u] = ((slot >> p.ps_log2) * p.Hk + h) * ((int64_t)1 << p.ps_log2) +
                   (slot & (((int64_t)1 << p.ps_log2) - 1));
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if constexpr (!E4M3) {
      if (place[u] >= 0)
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(cache) + place[u] * p.d + kE * part) = x[u][0];
    } else {
      constexpr uint32_t kInf = F16 ? 0x7C00u : 0x7F80u;
      const uint32_t w[8] = {x[u][0].x, x[u][0].y, x[u][0].z, x[u][0].w, x[u][1].x, x[u][1].y, x[u][1].z, x[u][1].w};
      uint32_t m2 = 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i) m2 = __vmaxu2(m2, w[i] & 0x7FFF7FFFu);
#pragma unroll
      for (int off = LANES / 2; off > 0; off >>= 1) m2 = __vmaxu2(m2, __shfl_xor_sync(0xFFFFFFFFu, m2, off));
      uint32_t top16 = max(m2 & 0xFFFFu, m2 >> 16);
      const bool odd = top16 >= kInf;   // the same in all threads of the row
      if (__any_sync(0xFFFFFFFFu, odd)) {
        // the largest finite pattern instead
        uint32_t fin = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t lo = w[i] & 0x7FFFu, hi = (w[i] >> 16) & 0x7FFFu;
          if (lo < kInf) fin = max(fin, lo);
          if (hi < kInf) fin = max(fin, hi);
        }
#pragma unroll
        for (int off = LANES / 2; off > 0; off >>= 1) fin = max(fin, __shfl_xor_sync(0xFFFFFFFFu, fin, off));
        top16 = fin;
      }
      const float top = F16 ? unpack2<true>(top16).x : __uint_as_float(top16 << 16);
      // top = (1 + m) 2^k: the smallest e with top <= 448 2^e = 1.75 2^(8 + e) is
      // k - 8, or one more where 1 + m > 1.75 (fp32-subnormal tops are under the floor)
      const uint32_t bits = __float_as_uint(top);
      int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
      e = e < -64 ? -64 : e;
      const float inv = __uint_as_float((uint32_t)(127 - e) << 23);   // 2^-e, exact
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float2 a = unpack2<F16>(w[2 * i]), b = unpack2<F16>(w[2 * i + 1]);
        if (odd) {   // infinities and NaN: stored as NaN
          const float nan = __int_as_float(0x7FC00000);
          a.x = fabsf(a.x) < INFINITY ? a.x : nan;
          a.y = fabsf(a.y) < INFINITY ? a.y : nan;
          b.x = fabsf(b.x) < INFINITY ? b.x : nan;
          b.y = fabsf(b.y) < INFINITY ? b.y : nan;
        }
        o[i] = (uint32_t)cvt_e4m3x2(a.x * inv, a.y * inv) | ((uint32_t)cvt_e4m3x2(b.x * inv, b.y * inv) << 16);
      }
      if (place[u] >= 0) {
        *reinterpret_cast<uint4*>(static_cast<uint8_t*>(cache) + place[u] * p.d + kE * part) =
            make_uint4(o[0], o[1], o[2], o[3]);
        if (part == 0) (is_v ? p.scale[1] : p.scale[0])[place[u]] = __uint_as_float((uint32_t)(127 + e) << 23);
      }
    }
  }
}

template <int LANES, int U, bool E4M3, bool F16>
cudaError_t launch_write_u(const WriteParams& p, cudaStream_t s) {
  const uint32_t per = 256 / LANES * U;
  return launch_pdl(true, kv_cache_write_kernel<LANES, U, E4M3, F16>, dim3((p.rows + per - 1) / per, 2), dim3(256), 0, s, p);
}

template <bool E4M3, bool F16>
cudaError_t launch_write(const WriteParams& p, cudaStream_t s) {
  const int lanes = p.d / (E4M3 ? 16 : 8);   // 1 .. 8 or 1 .. 16, rounded up to a power of two
  const bool many = p.rows >= kManyRows;
#define FA_WRITE_CASE(LL) \
  if (lanes <= LL) return many ? launch_write_u<LL, 2, E4M3, F16>(p, s) : launch_write_u<LL, 1, E4M3, F16>(p, s);
  FA_WRITE_CASE(1)
  FA_WRITE_CASE(2)
  FA_WRITE_CASE(4)
  FA_WRITE_CASE(8)
  if constexpr (!E4M3) {
    FA_WRITE_CASE(16)
  }
#undef FA_WRITE_CASE
  return cudaErrorInvalidValue;
}

// --------------------------------------------------------------------------
// attention against the cache
// --------------------------------------------------------------------------

constexpr int kMaxCtas = 152;
constexpr int kMaxWorkers = 12 * kMaxCtas;
constexpr int kRows = 16;                 // query rows of a unit
constexpr float kMoveThreshold = 8.0f;    // log2 units: the reference moves only past it

// Shared-memory layout, a ring of tiles for each warp. A tile is kKT keys: K,
// then V, each as the TMA writes it (16-bit: 64-column atoms of 128-byte rows;
// e4m3: one atom of D-byte rows), 128- or 64-byte swizzled; with e4m3 the scales
// of K and of V lie behind all rings (16 keys at a pitch of 64 bytes, or of 128
// where they come from two pages).
//
// Warps, keys of a tile and tiles of a ring, by the tile width D (64 or 128), the
// type and the kernel. A tile costs a warp its latency, 1 us or so, so the split
// over the GPU wants warps. 16-bit, d = 128, 12 x 16 keys x 2 against 6 x 32 x 2:
// the 64 sequences 101 and 113 us, 256 of 19381 tokens in all (20-200 each) 28.9 and
// 37.6, 16 of 381292 in all 240 and 240. e4m3, with twice the keys to a byte, 12
// warps of 32 keys x 2 against 8 x 32 x 3: the 16 sequences 161 and 174 us; at d =
// 64 with 64-key tiles, so that a step has as many bytes as at 128: 64 sequences of
// 151070 tokens in all 39 us, 46 with 12 x 32 x 4, 43 with 8 x 64 x 3. The warps of
// a cluster join their parts, and four of them with larger tiles do better: one
// sequence of 500 tokens 6.8 us with 4 x 32 x 3, 7.5 with 12 x 16 x 2, four of 4000
// 15.9 and 16.9.
struct Shape {
  int keys, warps, stages;
};
constexpr Shape cached_shape(int D, bool e4m3, bool whole) {
  if (e4m3) return whole ? Shape{32, 8, D == 128 ? 3 : 4} : Shape{D == 128 ? 32 : 64, 12, 2};
  if (whole) return D == 128 ? Shape{32, 4, 3} : Shape{32, 8, 3};
  return D == 128 ? Shape{16, 12, 2} : Shape{32, 12, 2};
}

template <int D, bool E4M3, bool WHOLE>
struct CachedLayout {
  static constexpr Shape kShape = cached_shape(D, E4M3, WHOLE);
  static constexpr int kKT = kShape.keys;
  static constexpr int kWarps = kShape.warps;
  static constexpr int kRowBytes = E4M3 ? D : 128;              // of a swizzle atom
  static constexpr int kAtoms = E4M3 ? 1 : D / 64;
  static constexpr int kAtomBytes = kKT * kRowBytes;
  static constexpr int kTileBytes = kAtoms * kAtomBytes;        // K or V
  static constexpr int kScaleBytes = E4M3 ? 8 * kKT : 0;        // K or V
  // stages start at multiples of 1024 bytes; the scales of all stages follow
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kStages = kShape.stages;
  static constexpr int kWarpBytes = kStages * kStageBytes;
  static constexpr int kScale = kWarps * kWarpBytes;
  // What a tile's scales do to its scores: worked out by every lane for its own
  // keys, or, with 64 keys, once per key and passed on through shared memory (per
  // warp, by pairs of keys: the factors and the log2 added, then the reciprocals).
  // 64 sequences of 151070 tokens in all at d = 64 39 us so and 42 without; at d =
  // 128, with 32 keys, the step through memory costs more than it saves (the 16
  // sequences 164 and 161 us).
  static constexpr bool kByKey = E4M3 && kKT == 64;
  static constexpr int kFactorBytes = kByKey ? 12 * kKT : 0;
  static constexpr int kFactors = kScale + kWarps * kStages * 2 * kScaleBytes;
  static constexpr int kBar = kFactors + kWarps * kFactorBytes;
  static constexpr int kMisc = kBar + 8 * kWarps * kStages;     // abort flag, -, wait limit, -
  static constexpr int kScan = kMisc + 16;                      // int64 [kWarps] totals, int64 [kWarps] starts, int [kWarps]
  static constexpr int kMl = (kScan + kWarps * 20 + 15) & ~15;  // (reference, sum) of kRows rows of each warp's part and of the CTA's
  static constexpr int kSmemBytes = kMl + (WHOLE ? (kWarps + 1) * kRows * 8 : 0);
  static constexpr uint32_t kTxBytes = 2u * kTileBytes + (E4M3 ? 2u * kKT * 4u : 0u);
  static_assert(kSmemBytes <= 232448, "shared memory budget");
};

struct CachedParams {
  const uint16_t* q;
  int64_t q_tok;
  const int32_t* table;
  const int32_t* lens;
  uint16_t* o;
  float* lse;
  float* part_o;       // [kMaxWorkers][2][kRows][D]
  float2* part_ml;     // [kMaxWorkers][2][kRows]: reference (log2), sum
  int2* info;          // [B Hk RT]: first and last worker of a (sequence, head, row tile) held in parts, or -1
  unsigned int* err;
  int B, Nq, Hq, Hk, G, d, R, RT;
  int num_pages, page_size, ps_log2, max_pages;
  float scale_log2;
  uint32_t wait_us, stall;
  int cluster;         // WHOLE: CTAs to a unit
};

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <bool F16>
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16) mma_f16(c, a, b0, b1);
  else mma_bf16(c, a, b0, b1);
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// two e4m3 values (16 bits) -> fp16x2, exact
__device__ __forceinline__ uint32_t e4m3_to_f16(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
  return r;
}

// byte offset of 16-byte chunk c of row r in a swizzled atom
template <int ROWB>
__device__ __forceinline__ uint32_t swz(int r, int c) {
  if constexpr (ROWB == 128) return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4));
  return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

__device__ __forceinline__ void tma_load_2d_w(uint32_t dst, const CUtensorMap* m, uint32_t bar, int c0, int c1) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];\n\t}"
      :: "r"(dst), "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1) : "memory");
}

// barrier of a cluster's CTAs (all threads), and two floats of CTA `rank`'s
// shared memory at this CTA's address
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float2 cluster_ld2(uint32_t addr, int rank) {
  float2 v;
  asm volatile(
      "{\n\t.reg .b32 a;\n\t"
      "mapa.shared::cluster.u32 a, %2, %3;\n\t"
      "ld.shared::cluster.v2.f32 {%0, %1}, [a];\n\t}"
      : "=f"(v.x), "=f"(v.y) : "r"(addr), "r"(rank) : "memory");
  return v;
}

// Walks the units of a range: tile j of n of (sequence b, sub = head * RT + row tile).
struct Walk {
  int b, sub, j, n, len;
};

// WHOLE: instead of cutting all units into ranges, a cluster of CTAs takes one
// (sequence, key/value head, row tile) and cuts its tiles among its warps; the
// parts meet in shared memory (a CTA's, then the cluster's), so there is neither
// a workspace nor a second kernel. For calls of few, short sequences.
template <int D, bool E4M3, bool F16, bool WHOLE>
__global__ void __launch_bounds__(32 * CachedLayout<D, E4M3, WHOLE>::kWarps, 1)
fa_cached_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                 const __grid_constant__ CUtensorMap tks, const __grid_constant__ CUtensorMap tvs,
                 const CachedParams p) {
  using L = CachedLayout<D, E4M3, WHOLE>;
  constexpr int KT = L::kKT, kWarps = L::kWarps;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  // (what is the same in all lanes of a warp comes from a shuffle, so that the
  // compiler knows it: the copies' operands are uniform registers)
  auto same = [](int v) -> int { return __shfl_sync(0xFFFFFFFFu, v, 0); };
  const int tid = threadIdx.x, warp = same(tid >> 5), lane = tid & 31;
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  volatile uint32_t* abort_flag = misc;
  Ctl ctl{p.err, abort_flag};
  if ((sbase & 1023u) != 0u) {   // uniform across the CTA: nothing has started yet
    if (tid == 0) {
      uint32_t dummy = 0;
      Ctl c0{p.err, &dummy};
      report_error(c0, kErrSmemAlign, 200);
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

  // ---- this warp's range of units
  const int SUB = p.Hk * p.RT;
  const int cap = p.max_pages << p.ps_log2;
  auto seq_len = [&](int b) -> int {
    const int n = p.lens[b];
    return n < 0 ? 0 : (n > cap ? cap : n);
  };
  auto tiles_of = [&](int len) -> int { return len > 0 ? (len + KT - 1) / KT : 1; };   // an empty sequence is one empty tile
  int me = 0, todo = 0;
  long long t0 = 0, total = 0;
  int workers = 0;
  Walk w0;
  if constexpr (WHOLE) {
    const int unit = (int)blockIdx.x / p.cluster, rank = (int)blockIdx.x % p.cluster;
    w0.b = unit / SUB;
    w0.sub = unit % SUB;
    w0.len = same(seq_len(w0.b));
    w0.n = tiles_of(w0.len);
    const int all = kWarps * p.cluster, mine = kWarps * rank + warp;
    w0.j = (int)((long long)w0.n * mine / all);
    todo = (int)((long long)w0.n * (mine + 1) / all) - w0.j;
    __syncthreads();   // (the barriers are initialised)
  } else {
    long long* tot = reinterpret_cast<long long*>(smem + L::kScan);
    long long* start_t = tot + kWarps;      // first unit of each warp's range, then the tiles of the sequences before it
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
    total = all * SUB;
    workers = (int)min((long long)(kWarps * gridDim.x), total);
    // neighbouring ranges go to different SMs, so that a small call spreads out
    me = warp * (int)gridDim.x + (int)blockIdx.x;
    auto range_start = [&](int w) -> long long { return total * w / workers; };
    t0 = me < workers ? range_start(me) : total;
    if (lane == 0) start_t[warp] = t0;
    __syncthreads();
    long long cum = before + incl - mine;   // tiles of the sequences before b_lo
    for (int b = b_lo; b < b_hi; ++b) {
      const long long lo = cum * SUB, hi = (cum += tiles_of(seq_len(b))) * SUB;
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
        if (start_t[w] >= lo && start_t[w] < hi) {
          start_b[w] = b;
          tot[w] = lo;
        }
    }
    __syncthreads();
    if (me >= workers) {
      grid_dep_launch();
      return;
    }
    todo = same((int)(range_start(me + 1) - t0));
    w0.b = same(start_b[warp]);
    w0.len = same(seq_len(w0.b));
    w0.n = tiles_of(w0.len);
    const long long rem = t0 - tot[warp];
    w0.sub = same((int)(rem / w0.n));
    w0.j = same((int)(rem % w0.n));
  }
  grid_dep_launch();   // the next kernel may be scheduled (it waits for this one's end)
  auto advance = [&](Walk& w) {
    if (++w.j < w.n) return;
    w.j = 0;
    if (++w.sub < SUB) return;
    w.sub = 0;
    if (++w.b < p.B) {
      w.len = same(seq_len(w.b));
      w.n = tiles_of(w.len);
    }
  };

  // ---- loads (warp-wide): piece i of a tile is one page's share of it. The page
  // numbers of a tile are read when the tile before it is issued.
  const uint32_t ring = sbase + (uint32_t)(warp * L::kWarpBytes);
  const uint32_t sring = sbase + L::kScale + (uint32_t)(warp * L::kStages * 2 * L::kScaleBytes);
  const int box = p.page_size < KT ? p.page_size : KT;     // keys of a piece
  const int pieces = KT / box;                             // 1, 2 or 4
  const int nowhere = p.num_pages * p.Hk;                  // a coordinate past the cache: reads as zeros
  int issued = 0;
  // page of lane i's piece of the tile, or -1
  auto page_of = [&](const Walk& w) -> int {
    const int key = w.j * KT + (lane & (KT / 16 - 1)) * box;
    return w.b < p.B && key < w.len ? p.table[(int64_t)w.b * p.max_pages + (key >> p.ps_log2)] : -1;
  };
  auto issue = [&](const Walk& w, int pages) {
    const int s = issued % L::kStages;
    ++issued;
    const int hk = w.sub / p.RT;
    mbar_arrive_expect_tx_w(bar(s), L::kTxBytes);
#pragma unroll 1
    for (int i = 0; i < pieces; ++i) {
      const int page = __shfl_sync(0xFFFFFFFFu, pages, i);
      const int z = page >= 0 && page < p.num_pages ? page * p.Hk + hk : nowhere;
      const int y = (w.j * KT + i * box) & (p.page_size - 1);
      const uint32_t dst = ring + (uint32_t)(s * L::kStageBytes + i * box * L::kRowBytes);
#pragma unroll
      for (int a = 0; a < L::kAtoms; ++a) tma_load_3d_w(dst + a * L::kAtomBytes, &tk, bar(s), 64 * a, y, z);
#pragma unroll
      for (int a = 0; a < L::kAtoms; ++a)
        tma_load_3d_w(dst + L::kTileBytes + a * L::kAtomBytes, &tv, bar(s), 64 * a, y, z);
      if constexpr (E4M3) {
        const uint32_t sd = sring + (uint32_t)(s * 2 * L::kScaleBytes + i * 128);
        tma_load_2d_w(sd, &tks, bar(s), y, z);
        tma_load_2d_w(sd + L::kScaleBytes, &tvs, bar(s), y, z);
      }
    }
  };

  Walk wi = w0;
  int pages = page_of(wi);
  // the next tile of the range, and the pages of the one after it
  auto issue_next = [&]() {
    const Walk w = wi;
    const int pg = pages;
    advance(wi);
    pages = page_of(wi);
    issue(w, pg);
  };
#pragma unroll 1
  for (int s = 0; s < L::kStages && s < todo; ++s) {
    if (p.stall != 0u && s >= 1) break;   // test of the timeout path: tile 1 never comes
    issue_next();
  }

  // ---- the tiles of the range
  const int g = lane >> 2, t4 = lane & 3;
  constexpr int kSteps = D / 16;
  uint32_t qf[kSteps][4];
  float o[D / 8][4];
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, qs[2];
#pragma unroll
  for (int n = 0; n < D / 8; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) o[n][i] = 0.f;
  Walk w = w0;
  bool fresh = true;              // the next tile starts a (sequence, head, row tile) for this warp
  bool from_start = false;        // ... and is its first
  bool ok = true;
#pragma unroll 1
  for (int u = 0; u < todo; ++u) {
    const int hk = w.sub / p.RT, rt = w.sub % p.RT;
    if (fresh) {
      fresh = false;
      from_start = w.j == 0;   // (WHOLE: a warp has tiles of one sequence only, and this runs once)
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[n][i] = 0.f;
      m[0] = m[1] = -INFINITY;
      l[0] = l[1] = 0.f;
      qs[0] = qs[1] = 1.f;
      const uint16_t* qp[2];
      bool live[2];
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int r = rt * kRows + g + 8 * hh;
        live[hh] = r < p.R;
        const int i = r / p.G;
        qp[hh] = p.q + ((int64_t)w.b * p.Nq + i) * p.q_tok + (hk * p.G + r % p.G) * p.d;
      }
      // A fragments: 16-bit, K step ks holds dims 16 ks + {2t, 2t+1, 2t+8, 2t+9};
      // e4m3, dims 16 ks + {4t .. 4t+3} (the order K's bytes come in)
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int hh = i & 1, hi = i >> 1;
          const int c = 16 * ks + (E4M3 ? 4 * t4 + 2 * hi : 2 * t4 + 8 * hi);
          qf[ks][i] = live[hh] && c < p.d ? *reinterpret_cast<const uint32_t*>(qp[hh] + c) : 0u;
        }
      if constexpr (E4M3 && !F16) {
        // bf16 -> fp16: each row is divided by a power of two that puts its
        // largest magnitude in [2^7, 2^8); what then lies under fp16's smallest
        // step is under 2^-31 of that largest magnitude
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
    }
    const int s = u % L::kStages;
    ok = bar_wait_warp(bar(s), (uint32_t)(u / L::kStages) & 1u, ctl, 201);
    if (!ok) break;
    const uint32_t sk = ring + (uint32_t)(s * L::kStageBytes), sv = sk + L::kTileBytes;
    const int left = w.len - w.j * KT;      // keys of the sequence from this tile on
    if (left < KT) {
      // rows of V past the sequence: whatever the page holds there (NaN times a
      // weight of zero is NaN) becomes zeros
      const int first = left < 0 ? 0 : left;
      constexpr int kChunks = L::kRowBytes / 16;
      uint8_t* vt = smem + (sv - sbase);
      for (int c = lane; c < (KT - first) * kChunks * L::kAtoms; c += 32) {
        const int row = first + (c / kChunks) % (KT - first);
        const int a = c / (kChunks * (KT - first));
        *reinterpret_cast<uint4*>(vt + a * L::kAtomBytes + row * L::kRowBytes + 16 * (c % kChunks)) =
            make_uint4(0u, 0u, 0u, 0u);
      }
      fence_proxy_async_smem();   // the ring slot is written by TMA again later
      __syncwarp();
    }

    [[maybe_unused]] float* f = reinterpret_cast<float*>(smem + L::kFactors + warp * L::kFactorBytes);   // (kByKey)
    [[maybe_unused]] const uint8_t* ss = smem + (sring - sbase) + s * 2 * L::kScaleBytes;
    // (16 keys of a page, or more of them in one piece)
    [[maybe_unused]] auto place = [&](int key) -> int { return box == 16 ? (key >> 4) * 128 + (key & 15) * 4 : key * 4; };
    // a value's scale of 0 becomes 2^-64 and its row of V zeros (a lane writes the
    // chunks first .. last - 1 of it); in a branch of the whole warp that seldom runs
    [[maybe_unused]] auto no_scale = [&](float& vs, int key, int first, int last) {
      if (vs == 0.f) {
        vs = 0x1p-64f;
        for (int c = first; c < last; ++c)
          *reinterpret_cast<uint4*>(smem + (sv - sbase) + key * L::kRowBytes + 16 * c) = make_uint4(0u, 0u, 0u, 0u);
      }
      fence_proxy_async_smem();   // (as above)
      __syncwarp();
    };
    if constexpr (L::kByKey) {
#pragma unroll
      for (int key = lane; key < KT; key += 32) {
        const float ks = *reinterpret_cast<const float*>(ss + place(key));
        float vs = key < left ? *reinterpret_cast<const float*>(ss + L::kScaleBytes + place(key)) : 1.f;
        if (__any_sync(0xFFFFFFFFu, vs == 0.f)) no_scale(vs, key, 0, L::kRowBytes / 16);
        const int at = 4 * (key >> 1) + (key & 1);
        f[at] = ks * p.scale_log2;
        f[at + 2] = __log2f(vs);
        f[2 * KT + key] = __fdividef(1.f, vs);
      }
      __syncwarp();
    }

    // S = Q K^T: sc[2 n + i] of key 8 n + 2 t4 + (i & 1), rows g (i < 2) and g + 8
    float sc[KT / 8][4];
#pragma unroll
    for (int n = 0; n < KT / 8; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) sc[n][i] = 0.f;
    if constexpr (!E4M3) {
      float sd[KT / 8][4];   // odd steps' sums: twice as many independent products
#pragma unroll
      for (int n = 0; n < KT / 8; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) sd[n][i] = 0.f;
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks)
#pragma unroll
        for (int kk = 0; kk < KT / 16; ++kk) {
          // four 8 x 8 matrices: keys 0-7 / 8-15 of the 16, dims 0-7 / 8-15 of the step
          uint32_t b[4];
          const int row = 16 * kk + (lane & 7) + 8 * (lane >> 4);
          const int chunk = 2 * (ks & 3) + ((lane >> 3) & 1);
          ldsm4(b, sk + (uint32_t)((ks >> 2) * L::kAtomBytes) + swz<L::kRowBytes>(row, chunk));
          mma16<F16>((ks & 1) ? sd[2 * kk] : sc[2 * kk], qf[ks], b[0], b[1]);
          mma16<F16>((ks & 1) ? sd[2 * kk + 1] : sc[2 * kk + 1], qf[ks], b[2], b[3]);
        }
#pragma unroll
      for (int n = 0; n < KT / 8; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[n][i] += sd[n][i];
    } else {
#pragma unroll
      for (int c4 = 0; c4 < kSteps / 4; ++c4)
#pragma unroll
        for (int n = 0; n < KT / 8; ++n) {
          // four 16-dim chunks of 8 keys; a lane gets 4 payloads of each
          uint32_t b[4];
          ldsm4(b, sk + swz<L::kRowBytes>(8 * n + (lane & 7), 4 * c4 + (lane >> 3)));
#pragma unroll
          for (int i = 0; i < 4; ++i)
            mma_f16(sc[n], qf[4 * c4 + i], e4m3_to_f16(b[i] & 0xFFFFu), e4m3_to_f16(b[i] >> 16));
        }
    }
    // scores in log2 units; with e4m3 plus log2 of the value's scale
    float ivs[KT / 8][2];
    if constexpr (E4M3) {
      [[maybe_unused]] float2 vs2[KT / 8];
      if constexpr (!L::kByKey) {
        float least = 1.f;
#pragma unroll
        for (int n = 0; n < KT / 8; ++n) {
          const int key = 8 * n + 2 * t4;
          vs2[n] = *reinterpret_cast<const float2*>(ss + L::kScaleBytes + place(key));
          if (key >= left) vs2[n].x = 1.f;       // past the sequence: any scale, the weight is zero
          if (key + 1 >= left) vs2[n].y = 1.f;
          least = fmin3(least, vs2[n].x, vs2[n].y);
        }
        // (eight lanes hold a key's scale and share its row's chunks out)
        if (__any_sync(0xFFFFFFFFu, least == 0.f))
#pragma unroll
          for (int n = 0; n < KT / 8; ++n) {
            const int key = 8 * n + 2 * t4, end = g < L::kRowBytes / 16 ? g + 1 : g;
            no_scale(vs2[n].x, key, g, end);
            no_scale(vs2[n].y, key + 1, g, end);
          }
      }
#pragma unroll
      for (int n = 0; n < KT / 8; ++n) {
        float4 fa;   // two keys' factors, then what is added
        if constexpr (L::kByKey) {
          fa = *reinterpret_cast<const float4*>(f + 4 * (4 * n + t4));
          const float2 iv = *reinterpret_cast<const float2*>(f + 2 * KT + 2 * (4 * n + t4));
          ivs[n][0] = iv.x;
          ivs[n][1] = iv.y;
        } else {
          const int key = 8 * n + 2 * t4;
          const float2 ks2 = *reinterpret_cast<const float2*>(ss + place(key));
          ivs[n][0] = __fdividef(1.f, vs2[n].x);
          ivs[n][1] = __fdividef(1.f, vs2[n].y);
          fa = make_float4(ks2.x * p.scale_log2, ks2.y * p.scale_log2, __log2f(vs2[n].x), __log2f(vs2[n].y));
        }
        sc[n][0] = fmaf(sc[n][0] * qs[0], fa.x, fa.z);
        sc[n][1] = fmaf(sc[n][1] * qs[0], fa.y, fa.w);
        sc[n][2] = fmaf(sc[n][2] * qs[1], fa.x, fa.z);
        sc[n][3] = fmaf(sc[n][3] * qs[1], fa.y, fa.w);
      }
    } else {
#pragma unroll
      for (int n = 0; n < KT / 8; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[n][i] *= p.scale_log2;
    }
    if (left - (p.Nq - 1) < KT) {
      // token i sees the first left - (Nq - 1 - i) keys from here
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int lim = left - (p.Nq - 1) + (rt * kRows + g + 8 * hh) / p.G;
#pragma unroll
        for (int n = 0; n < KT / 8; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (8 * n + 2 * t4 + i >= min(lim, left)) sc[n][2 * hh + i] = -INFINITY;
      }
    }
    // running reference: moved when a row's maximum passes it by more than 2^8
    float alpha[2] = {1.f, 1.f};
    bool move = false;
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      float mx = -INFINITY;
#pragma unroll
      for (int n = 0; n < KT / 8; ++n) mx = fmaxf(mx, fmaxf(sc[n][2 * hh], sc[n][2 * hh + 1]));
      mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
      if (mx > m[hh] + kMoveThreshold || (m[hh] == -INFINITY && mx > -INFINITY)) {
        alpha[hh] = m[hh] == -INFINITY ? 0.f : ex2(m[hh] - mx);
        m[hh] = mx;
        l[hh] *= alpha[hh];
        move = true;
      }
    }
    if (__any_sync(0xFFFFFFFFu, move)) {
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[n][i] *= alpha[i >> 1];
    }
    const float ref[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
#pragma unroll
    for (int n = 0; n < KT / 8; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sc[n][i] = ex2(sc[n][i] - ref[i >> 1]);
        l[i >> 1] += E4M3 ? sc[n][i] * ivs[n][i & 1] : sc[n][i];
      }
    // O += P V, 16 keys at a time; P goes to 16 bits (of the inputs' type, or
    // fp16 with e4m3: weights of at most 2^8 lose 2^-11 of themselves at most,
    // or 2^-25 next to a largest one of about 1)
#pragma unroll
    for (int kk = 0; kk < KT / 16; ++kk) {
      constexpr bool PF16 = E4M3 || F16;
      uint32_t a[4];
      a[0] = pack2<PF16>(sc[2 * kk][0], sc[2 * kk][1]);
      a[1] = pack2<PF16>(sc[2 * kk][2], sc[2 * kk][3]);
      a[2] = pack2<PF16>(sc[2 * kk + 1][0], sc[2 * kk + 1][1]);
      a[3] = pack2<PF16>(sc[2 * kk + 1][2], sc[2 * kk + 1][3]);
      const int row = 16 * kk + (lane & 15);
#pragma unroll
      for (int c = 0; c < kSteps; ++c) {
        // !E4M3: dims 16 c .. 16 c + 15 as two 8-dim chunks; E4M3: one 16-dim
        // chunk per matrix pair, so every second c loads two
        uint32_t b[4];
        if constexpr (!E4M3) {
          const int chunk = 2 * (c & 3) + (lane >> 4);
          ldsm4_t(b, sv + (uint32_t)((c >> 2) * L::kAtomBytes) + swz<L::kRowBytes>(row, chunk));
          mma16<F16>(o[2 * c], a, b[0], b[1]);
          mma16<F16>(o[2 * c + 1], a, b[2], b[3]);
        } else if ((c & 1) == 0) {
          ldsm4_t(b, sv + swz<L::kRowBytes>(row, c + (lane >> 4)));
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            // a word: payloads (key 2t, dims 2n and 2n + 1), (key 2t + 1, the same dims)
            const uint32_t lo = prmt(b[2 * i], 0u, 0x3120u), hi = prmt(b[2 * i + 1], 0u, 0x3120u);
            mma_f16(o[2 * (c + i)], a, e4m3_to_f16(lo & 0xFFFFu), e4m3_to_f16(hi & 0xFFFFu));        // even dims
            mma_f16(o[2 * (c + i) + 1], a, e4m3_to_f16(lo >> 16), e4m3_to_f16(hi >> 16));            // odd dims
          }
        }
      }
    }
    __syncwarp();   // every lane has read the tile: its place may be loaded again
    if (issued < todo && p.stall == 0u) issue_next();

    if (!WHOLE && (w.j == w.n - 1 || u == todo - 1)) {
      // the end of a (sequence, head, row tile), or of what this warp has of it
      fresh = true;
      const bool whole = from_start && w.j == w.n - 1;
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        l[hh] += __shfl_xor_sync(0xFFFFFFFFu, l[hh], 1);
        l[hh] += __shfl_xor_sync(0xFFFFFFFFu, l[hh], 2);
      }
      if (from_start && lane == 0) {
        int2 f = make_int2(-1, -1);
        if (!whole) {
          // this warp's range starts it; the last unit belongs to the last worker
          // whose range starts at or before it
          const long long last = t0 + u + (w.n - 1 - w.j);
          f = make_int2(me, (int)(((last + 1) * workers + total - 1) / total) - 1);
        }
        p.info[(int64_t)w.b * SUB + w.sub] = f;
      }
      const int slot = 2 * me + (from_start ? 1 : 0);
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int rr = g + 8 * hh, r = rt * kRows + rr;
        if (r >= p.R) continue;
        if (whole) {
          const int i = r / p.G, h = hk * p.G + r % p.G;
          const float inv = l[hh] > 0.f ? 1.f / l[hh] : (l[hh] == 0.f ? 0.f : l[hh]);
          uint16_t* op = p.o + (((int64_t)w.b * p.Nq + i) * p.Hq + h) * p.d;
          if constexpr (!E4M3) {
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
              if (8 * n < p.d)
                *reinterpret_cast<uint32_t*>(op + 8 * n + 2 * t4) = pack2<F16>(o[n][2 * hh] * inv, o[n][2 * hh + 1] * inv);
          } else {
#pragma unroll
            for (int c = 0; c < kSteps; ++c)
              if (16 * c < p.d)
                *reinterpret_cast<uint2*>(op + 16 * c + 4 * t4) =
                    make_uint2(pack2<F16>(o[2 * c][2 * hh] * inv, o[2 * c + 1][2 * hh] * inv),
                               pack2<F16>(o[2 * c][2 * hh + 1] * inv, o[2 * c + 1][2 * hh + 1] * inv));
          }
          if (t4 == 0)
            p.lse[((int64_t)w.b * p.Hq + h) * p.Nq + i] =
                l[hh] == 0.f ? -INFINITY : (m[hh] + log2f(l[hh])) * 0.69314718055994531f;
        } else {
          float* po = p.part_o + ((int64_t)slot * kRows + rr) * D;
          if constexpr (!E4M3) {
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
              *reinterpret_cast<float2*>(po + 8 * n + 2 * t4) = make_float2(o[n][2 * hh], o[n][2 * hh + 1]);
          } else {
#pragma unroll
            for (int c = 0; c < kSteps; ++c)
              *reinterpret_cast<float4*>(po + 16 * c + 4 * t4) =
                  make_float4(o[2 * c][2 * hh], o[2 * c + 1][2 * hh], o[2 * c][2 * hh + 1], o[2 * c + 1][2 * hh + 1]);
          }
          if (t4 == 0) p.part_ml[(int64_t)slot * kRows + rr] = make_float2(m[hh], l[hh]);
        }
      }
    }
    advance(w);
  }
  // every load issued has landed before the warp leaves (after a timeout)
  if (!ok && lane == 0) report_aborted(ctl);
  if (!ok && lane == 0)
    for (int s = 0; s < L::kStages && s < issued; ++s)
      drain_wait(bar(s), (uint32_t)((issued - 1 - s) / L::kStages) & 1u);
  if constexpr (WHOLE) {
    // every warp's part in its own ring (whose tiles have all been read), the
    // CTA's part behind warp 0's
    __syncwarp();
    constexpr int kCta = kRows * D * 4;
    static_assert(2 * kCta <= L::kWarpBytes, "a ring holds two parts");
    float2* mls = reinterpret_cast<float2*>(smem + L::kMl);   // [kWarps + 1][kRows]
    uint8_t* my = smem + warp * L::kWarpBytes;
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      l[hh] += __shfl_xor_sync(0xFFFFFFFFu, l[hh], 1);
      l[hh] += __shfl_xor_sync(0xFFFFFFFFu, l[hh], 2);
      const int rr = g + 8 * hh;
      float* po = reinterpret_cast<float*>(my) + rr * D;
      if constexpr (!E4M3) {
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
          *reinterpret_cast<float2*>(po + 8 * n + 2 * t4) = make_float2(o[n][2 * hh], o[n][2 * hh + 1]);
      } else {
#pragma unroll
        for (int c = 0; c < kSteps; ++c)
          *reinterpret_cast<float4*>(po + 16 * c + 4 * t4) =
              make_float4(o[2 * c][2 * hh], o[2 * c + 1][2 * hh], o[2 * c][2 * hh + 1], o[2 * c + 1][2 * hh + 1]);
      }
      if (t4 == 0) mls[warp * kRows + rr] = make_float2(m[hh], l[hh]);
    }
    __syncthreads();
    const int hk = w0.sub / p.RT, rt = w0.sub % p.RT;
    auto put = [&](int rr, int c, float a0, float a1, float M, float ls) {   // columns c, c + 1 of row rr
      const int r = rt * kRows + rr;
      if (r >= p.R) return;
      const int i = r / p.G, h = hk * p.G + r % p.G;
      const float inv = ls > 0.f ? 1.f / ls : (ls == 0.f ? 0.f : ls);
      if (c < p.d)
        *reinterpret_cast<uint32_t*>(p.o + (((int64_t)w0.b * p.Nq + i) * p.Hq + h) * p.d + c) = pack2<F16>(a0 * inv, a1 * inv);
      if (c == 0)
        p.lse[((int64_t)w0.b * p.Hq + h) * p.Nq + i] = ls == 0.f ? -INFINITY : (M + log2f(ls)) * 0.69314718055994531f;
    };
    // a thread joins two columns of a row at a time
    for (int x = tid; x < kRows * D / 2; x += 32 * kWarps) {
      const int rr = x / (D / 2), c = 2 * (x % (D / 2));
      if (rt * kRows + rr >= p.R) break;   // (rows ascend with x)
      float M = -INFINITY;
#pragma unroll
      for (int k = 0; k < kWarps; ++k)
        M = fmaxf(M, mls[k * kRows + rr].x);
      const float ref = M == -INFINITY ? 0.f : M;
      float ls = 0.f, a0 = 0.f, a1 = 0.f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const float2 ml = mls[k * kRows + rr];
        const float2 v = *reinterpret_cast<const float2*>(smem + k * L::kWarpBytes + (rr * D + c) * 4);
        const float f = ex2(ml.x - ref);
        ls = fmaf(f, ml.y, ls);
        a0 = fmaf(f, v.x, a0);
        a1 = fmaf(f, v.y, a1);
      }
      if (p.cluster == 1) {
        put(rr, c, a0, a1, M, ls);
      } else {
        *reinterpret_cast<float2*>(smem + kCta + (rr * D + c) * 4) = make_float2(a0, a1);
        if (c == 0) mls[kWarps * kRows + rr] = make_float2(M, ls);
      }
    }
    if (p.cluster > 1) {
      cluster_sync();
      // the CTAs share the rows out; each reads the others' parts of its rows
      const int rank = (int)blockIdx.x % p.cluster;
      for (int x = tid;; x += 32 * kWarps) {
        const int rr = rank + p.cluster * (x / (D / 2)), c = 2 * (x % (D / 2));
        if (rr >= kRows || rt * kRows + rr >= p.R) break;
        float M = -INFINITY;
        for (int k = 0; k < p.cluster; ++k) M = fmaxf(M, cluster_ld2(sbase + L::kMl + 8 * (kWarps * kRows + rr), k).x);
        const float ref = M == -INFINITY ? 0.f : M;
        float ls = 0.f, a0 = 0.f, a1 = 0.f;
        for (int k = 0; k < p.cluster; ++k) {
          const float2 ml = cluster_ld2(sbase + L::kMl + 8 * (kWarps * kRows + rr), k);
          const float2 v = cluster_ld2(sbase + kCta + (rr * D + c) * 4, k);
          const float f = ex2(ml.x - ref);
          ls = fmaf(f, ml.y, ls);
          a0 = fmaf(f, v.x, a0);
          a1 = fmaf(f, v.y, a1);
        }
        put(rr, c, a0, a1, M, ls);
      }
      cluster_sync();   // no CTA leaves while another reads its part
    }
  }
}

// Joins the parts of a query row. m is a part's reference, l its sum:
//   O = sum_k 2^(m_k - M) O_k / sum_k 2^(m_k - M) l_k,  M = max m_k.
// WARPS warps share a row's parts out (a lane holds D / 32 columns, and the
// columns of kAhead parts are on their way before their weights are known); with
// WARPS = 1 a block of four warps joins four rows. The rows of one launch have
// about as many parts each as there are workers to a (sequence, head, row tile):
// from 8 kManyParts on 16 warps take a row, so that no warp walks a long list (one
// sequence of 32768 tokens, 228 parts a row: the call takes 29.5 us so, 37.4 with
// four warps), from kManyParts on four (the 16 sequences in e4m3, 14 parts: 161 us,
// 164 with one, 166 with 16), and below it one (256 sequences of 19381 tokens in all:
// 28.9 us, against 35.6 with a block of four).
constexpr int kManyParts = 8;

template <int D, bool F16, int WARPS>
__global__ void __launch_bounds__(WARPS == 1 ? 128 : 32 * WARPS) fa_cached_join_kernel(const CachedParams p) {
  constexpr int C = D / 32, kAhead = 8;
  __shared__ float sm_o[WARPS == 1 ? 1 : WARPS][D];
  __shared__ float2 sm_ml[WARPS];
  grid_dep_wait();   // the parts are complete
  const int warp = (int)threadIdx.x >> 5, lane = (int)threadIdx.x & 31;
  const unsigned row = WARPS == 1 ? blockIdx.x * 4u + (unsigned)warp : blockIdx.x;   // over [B][Hq][Nq]
  const int per_b = p.Hq * p.Nq;
  if (row >= (unsigned)(p.B * per_b)) return;
  const int b = (int)(row / (unsigned)per_b), x = (int)(row % (unsigned)per_b);
  const int h = x / p.Nq, i = x % p.Nq;
  const int hk = h / p.G, r = i * p.G + h % p.G;
  const int2 f = p.info[((int64_t)b * p.Hk + hk) * p.RT + r / kRows];
  // -1: written whole (or, after a timeout, nothing to join)
  if (f.x < 0 || f.y <= f.x || f.y >= kMaxWorkers) return;
  const int rr = r % kRows, parts = f.y - f.x + 1;
  auto at = [&](int k) -> int64_t { return (int64_t)(2 * (f.x + k) + (k == 0 ? 1 : 0)) * kRows + rr; };
  // this warp's parts k0, k0 + step, ..., a lane looking after the weight of one
  // of 32 of them, kAhead parts' columns on their way at a time
  const int k0 = WARPS == 1 ? 0 : warp, step = WARPS;
  const int mine = k0 < parts ? (parts - k0 + step - 1) / step : 0;
  float M = -INFINITY, l = 0.f, acc[C];
#pragma unroll
  for (int c = 0; c < C; ++c) acc[c] = 0.f;
  for (int base = 0; base < mine; base += 32) {
    const int n = min(32, mine - base);
    const float2 ml = lane < n ? p.part_ml[at(k0 + step * (base + lane))] : make_float2(-INFINITY, 0.f);
    // (the first columns are on their way while the weights are worked out)
    float v[kAhead][C];
    auto load = [&](int from) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (from + k < n) {
          const float* po = p.part_o + at(k0 + step * (base + from + k)) * D + C * lane;
          if constexpr (C == 4) {
            const float4 x4 = *reinterpret_cast<const float4*>(po);
            v[k][0] = x4.x;
            v[k][1] = x4.y;
            v[k][C - 2] = x4.z;
            v[k][C - 1] = x4.w;
          } else {
            const float2 x2 = *reinterpret_cast<const float2*>(po);
            v[k][0] = x2.x;
            v[k][1] = x2.y;
          }
        }
    };
    load(0);
    float mx = ml.x;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, off));
    const float Mn = fmaxf(M, mx), ref = Mn == -INFINITY ? 0.f : Mn;
    const float old = ex2(M - ref), wt = ex2(ml.x - ref);
    M = Mn;
    float ls = wt * ml.y;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) ls += __shfl_xor_sync(0xFFFFFFFFu, ls, off);
    l = fmaf(l, old, ls);
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] *= old;
    for (int from = 0; from < n; from += kAhead) {
      if (from > 0) load(from);
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const float w = __shfl_sync(0xFFFFFFFFu, wt, from + k);
        if (from + k < n) {
#pragma unroll
          for (int c = 0; c < C; ++c) acc[c] = fmaf(w, v[k][c], acc[c]);
        }
      }
    }
  }
  uint16_t* op = p.o + (((int64_t)b * p.Nq + i) * p.Hq + h) * p.d;
  float* lp = p.lse + ((int64_t)b * p.Hq + h) * p.Nq + i;
  if constexpr (WARPS > 1) {
#pragma unroll
    for (int c = 0; c < C; ++c) sm_o[warp][C * lane + c] = acc[c];
    if (lane == 0) sm_ml[warp] = make_float2(M, l);
    __syncthreads();
    if (warp > 0) return;
    float2 ml = lane < WARPS ? sm_ml[lane] : make_float2(-INFINITY, 0.f);
    M = ml.x;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, off));
    const float wt = ex2(ml.x - (M == -INFINITY ? 0.f : M));
    l = wt * ml.y;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, off);
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] = 0.f;
#pragma unroll
    for (int k = 0; k < WARPS; ++k) {
      const float w = __shfl_sync(0xFFFFFFFFu, wt, k);
#pragma unroll
      for (int c = 0; c < C; ++c) acc[c] = fmaf(w, sm_o[k][C * lane + c], acc[c]);
    }
  }
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
  if (C * lane < p.d) {
#pragma unroll
    for (int c = 0; c < C; c += 2)
      *reinterpret_cast<uint32_t*>(op + C * lane + c) = pack2<F16>(acc[c] * inv, acc[c + 1] * inv);
  }
  if (lane == 0) *lp = l == 0.f ? -INFINITY : (M + log2f(l)) * 0.69314718055994531f;
}

struct CachedWorkspace {
  size_t o_off, ml_off, info_off, total;
};

CachedWorkspace cached_workspace_layout(int B, int Nq, int Hq, int Hk, int d) {
  auto al = [](size_t x) { return (x + 255) & ~size_t(255); };
  const size_t D = d <= 64 ? 64 : 128;
  const size_t RT = ((size_t)Nq * (Hq / Hk) + kRows - 1) / kRows;
  CachedWorkspace w;
  w.o_off = 0;
  w.ml_off = al((size_t)kMaxWorkers * 2 * kRows * D * sizeof(float));
  w.info_off = al(w.ml_off + (size_t)kMaxWorkers * 2 * kRows * sizeof(float2));
  w.total = al(w.info_off + (size_t)B * Hk * RT * sizeof(int2));
  return w;
}

// The number of CTAs (a cluster) that take a (sequence, head, row tile) together,
// or 0 where the split over all warps of the GPU serves better. As many as the
// card holds at once (15 clusters of 8, 36 of 4, 76 of 2: a cluster lives within
// one group of SMs) and as have a tile for each warp. A tile costs a warp about
// 0.9 us, so that is taken while a warp gets at most 16 tiles of the longest
// sequence that the table has room for, 12 where less than half of the card works
// (us, so and, with a table of 262144 keys, split; inputs not in L2, 8 key/value
// heads, d = 128: 1 x 500 bf16 7.1 and 8.8, 1 x 4000 10.0 and 11.9, 1 x 8000 14.1 and
// 14.7, 16 x 500 11.8 and 16.3, 4 x 8000 26.7 and 31.4; e4m3 1 x 4000 9.2 and 10.9,
// 1 x 8000 12.7 and 14.5, 4 x 8000 21.1 and 24.5). Towards the end of a single
// sequence's range the split has become the faster one, since its join loads parts
// early: 1 x 12000 bf16 18.1 and 16.8; e4m3 1 x 16000 19.1 and 18.3, 1 x 24000 25.4
// and 21.3.
int whole_cluster(long long units, long long tiles, int warps) {
  int c = 8;
  const auto most = [](int cc) { return cc == 8 ? 15 : cc == 4 ? 36 : kMaxCtas / cc; };
  while (c > 1 && (units > most(c) || tiles <= (long long)warps * (c / 2))) c /= 2;
  if (units > most(c)) return 0;
  const int per_warp = 2 * units * c > kMaxCtas ? 16 : 12;
  return tiles <= (long long)per_warp * warps * c ? c : 0;
}

int cached_whole(int B, int Nq, int Hq, int Hk, int d, int page_size, int max_pages, bool e4m3) {
  const long long units = (long long)B * Hk * (((long long)Nq * (Hq / Hk) + kRows - 1) / kRows);
  const Shape sh = cached_shape(d <= 64 ? 64 : 128, e4m3, true);
  return whole_cluster(units, ((long long)max_pages * page_size + sh.keys - 1) / sh.keys, sh.warps);
}

fa_status check_cached_shape(int B, int Nq, int Hq, int Hk, int d) {
  if (B < 1 || Nq < 1 || Hk < 1 || Hq < 1 || Hq % Hk != 0) return FA_ERR_INVALID_ARG;
  if (d < 8 || d > 128 || d % 8 != 0) return FA_ERR_UNSUPPORTED;
  const double units = (double)B * Nq * Hq;
  if (units > 1073741824.0) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

// page sizes the kernels take: 16 .. 256, powers of two; the exponent, or -1
int page_log2(int page_size) {
  for (int k = 4; k <= 8; ++k)
    if (page_size == (1 << k)) return k;
  return -1;
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

template <int D, bool E4M3, bool F16>
cudaError_t launch_cached_d(const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& tks,
                            const CUtensorMap& tvs, CachedParams p, cudaStream_t s) {
  using L = CachedLayout<D, E4M3, false>;
  using LW = CachedLayout<D, E4M3, true>;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static PerDeviceOnce smem_set;
  e = once_per_device(smem_set, dev, [] {
    const cudaError_t e1 = cudaFuncSetAttribute(fa_cached_kernel<D, E4M3, F16, false>,
                                                cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmemBytes);
    return e1 != cudaSuccess ? e1
                             : cudaFuncSetAttribute(fa_cached_kernel<D, E4M3, F16, true>,
                                                    cudaFuncAttributeMaxDynamicSharedMemorySize, LW::kSmemBytes);
  });
  if (e != cudaSuccess) return e;
  if (p.cluster > 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.B * p.Hk * p.RT * p.cluster));
    cfg.blockDim = dim3(32 * LW::kWarps);
    cfg.dynamicSmemBytes = LW::kSmemBytes;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)p.cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, fa_cached_kernel<D, E4M3, F16, true>, tk, tv, tks, tvs, p);
  }
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  // one CTA per SM, fewer when even full sequences have fewer units
  const double most = (double)p.B * p.Hk * p.RT * (((double)p.max_pages * p.page_size + L::kKT - 1) / L::kKT);
  int ctas = sms < kMaxCtas ? sms : kMaxCtas;
  if (most < ctas) ctas = most < 1.0 ? 1 : (int)most;
  e = launch_pdl(true, fa_cached_kernel<D, E4M3, F16, false>, dim3((unsigned)ctas), dim3(32 * L::kWarps), L::kSmemBytes, s, tk, tv,
                 tks, tvs, p);
  if (e != cudaSuccess) return e;
  const unsigned rows = (unsigned)(p.B * p.Hq * p.Nq);
  const long long units = (long long)p.B * p.Hk * p.RT, workers = (long long)L::kWarps * ctas;
  if (units * 8 * kManyParts <= workers)
    return launch_pdl(true, fa_cached_join_kernel<D, F16, 16>, dim3(rows), dim3(512), 0, s, p);
  if (units * kManyParts <= workers)
    return launch_pdl(true, fa_cached_join_kernel<D, F16, 4>, dim3(rows), dim3(128), 0, s, p);
  return launch_pdl(true, fa_cached_join_kernel<D, F16, 1>, dim3((rows + 3) / 4), dim3(128), 0, s, p);
}

}  // namespace

}  // namespace fa

using namespace fa;

extern "C" {

fa_status flash_attn_kv_cache_write(const void* K, const void* V, int64_t k_token_stride, int64_t k_head_stride,
                                    int64_t v_token_stride, int64_t v_head_stride, const int64_t* slots, int T,
                                    int Hk, int d, void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                                    int num_pages, int page_size, int cache_type, const fa_options* options,
                                    void* stream) {
  const bool e4m3 = cache_type == FA_CACHE_E4M3;
  if (T < 0 || Hk < 1 || num_pages < 1) return FA_ERR_INVALID_ARG;
  if (!e4m3 && cache_type != FA_CACHE_16BIT) return FA_ERR_UNSUPPORTED;
  if (d < 8 || d > 128 || d % (e4m3 ? 16 : 8) != 0) return FA_ERR_UNSUPPORTED;
  const int pl = page_log2(page_size);
  if (pl < 0) return FA_ERR_UNSUPPORTED;
  if ((double)T * Hk > kMaxWriteRows || Hk > kMaxWriteHeads) return FA_ERR_UNSUPPORTED;
  bool f16 = false, flash_only = false;
  int st = internal_read_options(options, &f16, &flash_only);
  if (st != FA_OK) return static_cast<fa_status>(st);
  if (flash_only) return FA_ERR_UNSUPPORTED;
  if (k_cache == nullptr || v_cache == nullptr || !aligned(k_cache, 16) || !aligned(v_cache, 16))
    return FA_ERR_INVALID_ARG;
  if (e4m3 ? (k_scale == nullptr || v_scale == nullptr || !aligned(k_scale, 16) || !aligned(v_scale, 16))
           : (k_scale != nullptr || v_scale != nullptr))
    return FA_ERR_INVALID_ARG;
  if (T == 0) return FA_OK;
  if (K == nullptr || V == nullptr || slots == nullptr || !aligned(K, 16) || !aligned(V, 16) || !aligned(slots, 8) ||
      ((k_token_stride | k_head_stride | v_token_stride | v_head_stride) & 7) != 0 || k_token_stride <= 0 ||
      k_head_stride <= 0 || v_token_stride <= 0 || v_head_stride <= 0)
    return FA_ERR_INVALID_ARG;
  unsigned int* err = nullptr;
  if ((st = internal_device_error_word(&err)) != FA_OK) return static_cast<fa_status>(st);
  WriteParams p{};
  p.src[0] = static_cast<const uint16_t*>(K);
  p.src[1] = static_cast<const uint16_t*>(V);
  p.tok[0] = k_token_stride;
  p.tok[1] = v_token_stride;
  p.head[0] = k_head_stride;
  p.head[1] = v_head_stride;
  p.slots = slots;
  p.cache[0] = k_cache;
  p.cache[1] = v_cache;
  p.scale[0] = k_scale;
  p.scale[1] = v_scale;
  p.rows = (uint32_t)T * (uint32_t)Hk;
  p.Hk = (uint32_t)Hk;
  p.magic = write_magic(Hk);
  p.d = d;
  p.ps_log2 = pl;
  p.places = (int64_t)num_pages * page_size;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = !e4m3 ? launch_write<false, false>(p, s)
                        : f16 ? launch_write<true, true>(p, s)
                              : launch_write<true, false>(p, s);
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

size_t flash_attn_cached_workspace_size(int B, int Nq, int Hq, int Hk, int d) {
  if (check_cached_shape(B, Nq, Hq, Hk, d) != FA_OK) return 0;
  return cached_workspace_layout(B, Nq, Hq, Hk, d).total;
}

int flash_attn_cached_needs_workspace(int B, int Nq, int Hq, int Hk, int d, int page_size, int max_pages,
                                      int cache_type) {
  if (check_cached_shape(B, Nq, Hq, Hk, d) != FA_OK || page_log2(page_size) < 0 || max_pages < 1) return 1;
  return cached_whole(B, Nq, Hq, Hk, d, page_size, max_pages, cache_type == FA_CACHE_E4M3) > 0 ? 0 : 1;
}

fa_status flash_attn_cached_fwd(const void* Q, int64_t q_token_stride, const void* k_cache, const void* v_cache,
                                const float* k_scale, const float* v_scale, const int32_t* block_table,
                                const int32_t* seq_lens, void* O, float* LSE, int B, int Nq, int Hq, int Hk, int d,
                                int num_pages, int page_size, int max_pages, float scale, int cache_type,
                                const fa_options* options, void* workspace, size_t workspace_bytes, void* stream) {
  const bool e4m3 = cache_type == FA_CACHE_E4M3;
  fa_status st = check_cached_shape(B, Nq, Hq, Hk, d);
  if (st != FA_OK) return st;
  if (num_pages < 1 || max_pages < 1 || !std::isfinite(scale) || scale <= 0.f) return FA_ERR_INVALID_ARG;
  if (!e4m3 && cache_type != FA_CACHE_16BIT) return FA_ERR_UNSUPPORTED;
  if (e4m3 && d % 16 != 0) return FA_ERR_UNSUPPORTED;
  const int pl = page_log2(page_size);
  if (pl < 0) return FA_ERR_UNSUPPORTED;
  // page * Hk is a TMA coordinate, lengths and key numbers are 32-bit
  if ((double)num_pages * Hk > 2147480000.0 || (double)max_pages * page_size > 1073741824.0) return FA_ERR_UNSUPPORTED;
  bool f16 = false, record = false;
  uint32_t wait_us = 0, stall = 0;
  int sr = internal_read_check_options(options, &f16, &record, &wait_us, &stall);
  if (sr != FA_OK) return static_cast<fa_status>(sr);
  if (record) return FA_ERR_UNSUPPORTED;
  const void* ptrs[] = {Q, k_cache, v_cache, O, LSE, block_table, seq_lens};
  for (const void* x : ptrs)
    if (x == nullptr) return FA_ERR_INVALID_ARG;
  if (!aligned(Q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(O, 16) || !aligned(LSE, 4) ||
      !aligned(block_table, 4) || !aligned(seq_lens, 4))
    return FA_ERR_INVALID_ARG;
  if ((q_token_stride & 7) != 0 || q_token_stride < (int64_t)Hq * d) return FA_ERR_INVALID_ARG;
  if (e4m3 ? (k_scale == nullptr || v_scale == nullptr || !aligned(k_scale, 16) || !aligned(v_scale, 16))
           : (k_scale != nullptr || v_scale != nullptr))
    return FA_ERR_INVALID_ARG;
  const CachedWorkspace w = cached_workspace_layout(B, Nq, Hq, Hk, d);
  const int cluster = cached_whole(B, Nq, Hq, Hk, d, page_size, max_pages, e4m3);
  if (!(cluster > 0 && workspace == nullptr) &&   // (such calls use none)
      (workspace == nullptr || !aligned(workspace, 256) || workspace_bytes < w.total))
    return FA_ERR_WORKSPACE;
  unsigned int* err = nullptr;
  if ((sr = internal_device_error_word(&err)) != FA_OK) return static_cast<fa_status>(sr);

  const int D = d <= 64 ? 64 : 128;
  const int keys = cached_shape(D, e4m3, cluster > 0).keys;
  const uint32_t box_keys = (uint32_t)(page_size < keys ? page_size : keys);
  CUtensorMap tk, tv, tks, tvs;
  {
    const uint64_t es = e4m3 ? 1 : 2;
    const uint64_t dims[3] = {(uint64_t)d, (uint64_t)page_size, (uint64_t)num_pages * Hk};
    const uint64_t strides[2] = {d * es, (uint64_t)page_size * d * es};
    const uint32_t box[3] = {(uint32_t)(e4m3 ? D : 64), box_keys, 1};
    const CUtensorMapDataType ty = e4m3  ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                         : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const CUtensorMapSwizzle sw = e4m3 && D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
    if (internal_tensor_map(&tk, ty, 3, k_cache, dims, strides, box, sw) ||
        internal_tensor_map(&tv, ty, 3, v_cache, dims, strides, box, sw))
      return FA_ERR_CUDA;
    const uint64_t sdims[2] = {(uint64_t)page_size, (uint64_t)num_pages * Hk};
    const uint64_t sstr[1] = {(uint64_t)page_size * 4};
    const uint32_t sbox[2] = {box_keys, 1};
    tks = tk;
    tvs = tv;
    if (e4m3 &&
        (internal_tensor_map(&tks, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, k_scale, sdims, sstr, sbox,
                             CU_TENSOR_MAP_SWIZZLE_NONE) ||
         internal_tensor_map(&tvs, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, v_scale, sdims, sstr, sbox,
                             CU_TENSOR_MAP_SWIZZLE_NONE)))
      return FA_ERR_CUDA;
  }
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  CachedParams p{};
  p.q = static_cast<const uint16_t*>(Q);
  p.q_tok = q_token_stride;
  p.table = block_table;
  p.lens = seq_lens;
  p.o = static_cast<uint16_t*>(O);
  p.lse = LSE;
  p.part_o = reinterpret_cast<float*>(ws + w.o_off);
  p.part_ml = reinterpret_cast<float2*>(ws + w.ml_off);
  p.info = reinterpret_cast<int2*>(ws + w.info_off);
  p.err = err;
  p.B = B;
  p.Nq = Nq;
  p.Hq = Hq;
  p.Hk = Hk;
  p.G = Hq / Hk;
  p.d = d;
  p.R = Nq * p.G;
  p.RT = (p.R + kRows - 1) / kRows;
  p.num_pages = num_pages;
  p.page_size = page_size;
  p.ps_log2 = pl;
  p.max_pages = max_pages;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.wait_us = wait_us;
  p.stall = stall;
  p.cluster = cluster;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaErrorInvalidValue;
#define FA_CACHED_CASE(DD, EE, FF) \
  if (D == DD && e4m3 == EE && f16 == FF) e = launch_cached_d<DD, EE, FF>(tk, tv, tks, tvs, p, s);
  FA_CACHED_CASE(64, false, false)
  FA_CACHED_CASE(64, false, true)
  FA_CACHED_CASE(64, true, false)
  FA_CACHED_CASE(64, true, true)
  FA_CACHED_CASE(128, false, false)
  FA_CACHED_CASE(128, false, true)
  FA_CACHED_CASE(128, true, false)
  FA_CACHED_CASE(128, true, true)
#undef FA_CACHED_CASE
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
