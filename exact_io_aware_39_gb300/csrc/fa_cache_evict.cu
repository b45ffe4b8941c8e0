// A paged cache shortened to the tokens with the most accumulated attention
// (flash_attn_kv_cache_evict in flash_attn_cache.h), for sm_103a, in two kernels:
// one finds the tokens that stay, for each sequence and key/value head by itself,
// the other copies their rows to the pages of the new table.
//
// The selection: a weight >= 0 orders as its bits do, so the weight of the last
// token that stays is found from the top, 11, 11 and 10 bits at a time (a histogram
// of the tokens that agree with what is known so far, summed from above), and a pass
// over the tokens in order then lists those over it and as many of those equal to
// it as are missing, the first ones. Eleven bits are the exponent and two more, so
// that even the first histogram's counts spread over some forty places. A cluster of
// up to 8 CTAs shares a (sequence, head): each gathers its share of the weights into
// shared memory once, the histograms are added up through distributed shared
// memory. (The whole call, with one CTA that reads the weights again from L2 in each of
// five passes of 8 bits, and so: 2 sequences of 65536 tokens, 8 heads, d = 128, to a
// quarter 165 and 53 us; 32 of 512-8192 to 1024 tokens 67 and 55.)
//
// The copy is bound by memory: it reads and writes each kept row once; a scale or a
// weight, 4 bytes from a place of its own, costs a sector of 32.
#include "flash_attn_cache.h"
#include "fa_common.cuh"
#include "fa_ptx.cuh"

namespace fa {

namespace {

struct EvictParams {
  uint8_t* cache[2];        // K, V
  float* scale[2];          // or null
  float* weights;
  const int32_t* table;     // [B, max_pages]
  const int32_t* lens;
  const int32_t* new_table; // [B, new_pages]
  int32_t* new_lens;
  int32_t* kept;            // [B, Hk, budget]
  int B, Hk, row_bytes, num_pages, page_size, ps_log2, max_pages, new_pages, budget, recent;
};

constexpr int kSelectThreads = 512, kBins = 2048, kMaxCluster = 8;
constexpr int kMaxKeys = 40960;   // weights of a CTA's share that are kept in shared memory (160 KB)
constexpr int kCopyThreads = 256, kCopyBytes = 32768;

__device__ __forceinline__ int evict_len(const EvictParams& p, int b) {
  const int n = p.lens[b], cap = p.max_pages << p.ps_log2;
  return n < 0 ? 0 : (n > cap ? cap : n);
}

// Place of token j of head hk in a table's pages ([num_pages, Hk, page_size]), or -1.
__device__ __forceinline__ int64_t evict_place(const EvictParams& p, const int32_t* row, int j, int hk) {
  const int page = row[j >> p.ps_log2];
  return page >= 0 && page < p.num_pages ? ((int64_t)page * p.Hk + hk) * p.page_size + (j & (p.page_size - 1)) : -1;
}

__device__ __forceinline__ uint32_t cluster_address(uint32_t addr, int rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  return a;
}
__device__ __forceinline__ int2 cluster_ld2(uint32_t addr, int rank) {
  int2 v;
  asm volatile("ld.shared::cluster.v2.s32 {%0, %1}, [%2];"
               : "=r"(v.x), "=r"(v.y) : "r"(cluster_address(addr, rank)) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// A block's sum of v over the threads before this one, and over all of them.
constexpr int kSelectWarps = kSelectThreads / 32;
__device__ __forceinline__ int2 scan_warp(int2 x) {   // inclusive
  const int lane = (int)threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xFFFFFFFFu, x.x, o), b = __shfl_up_sync(0xFFFFFFFFu, x.y, o);
    if (lane >= o) {
      x.x += a;
      x.y += b;
    }
  }
  return x;
}
__device__ __forceinline__ int2 block_before(int2 v, int2 (&sums)[kSelectWarps], int2* all) {
  const int warp = (int)threadIdx.x >> 5, lane = (int)threadIdx.x & 31;
  const int2 x = scan_warp(v);
  __syncthreads();   // (the last call's sums have been read)
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  const int2 own = lane < kSelectWarps ? sums[lane] : make_int2(0, 0);
  const int2 upto = scan_warp(own);
  *all = make_int2(__shfl_sync(0xFFFFFFFFu, upto.x, 31), __shfl_sync(0xFFFFFFFFu, upto.y, 31));
  return make_int2(__shfl_sync(0xFFFFFFFFu, upto.x - own.x, warp) + x.x - v.x,
                   __shfl_sync(0xFFFFFFFFu, upto.y - own.y, warp) + x.y - v.y);
}

// A cluster of `ctas` CTAs per (sequence, head); `room` weights of each in shared
// memory.
__global__ void __launch_bounds__(kSelectThreads, 2) evict_select_kernel(const EvictParams p, const int ctas, const int room) {
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ __align__(8) int hist[3][kBins];
  __shared__ int2 sums[kSelectWarps];
  __shared__ __align__(8) int2 counts;   // this CTA's tokens over the threshold, equal to it
  __shared__ int s_digit, s_need;
  const int tid = threadIdx.x;
  for (int i = tid; i < 3 * kBins; i += kSelectThreads) hist[i / kBins][i % kBins] = 0;
  __syncthreads();
  grid_dep_wait();
  grid_dep_launch();
  const int bh = (int)blockIdx.x / ctas, rank = (int)blockIdx.x % ctas;
  const int b = bh / p.Hk, hk = bh % p.Hk;
  const int n = evict_len(p, b);
  int32_t* kept = p.kept + (int64_t)bh * p.budget;
  const int all = ctas * kSelectThreads, me = rank * kSelectThreads + tid;
  if (n <= p.budget) {   // (the same in the whole cluster)
    for (int j = me; j < p.budget; j += all) kept[j] = j < n ? j : -1;
    return;
  }
  const int older = n - p.recent, want = p.budget - p.recent;   // 0 <= want < older
  for (int i = me; i < p.recent; i += all) kept[want + i] = older + i;
  if (want == 0) return;
  // this CTA's tokens lo .. lo + mine - 1
  const int32_t* row = p.table + (int64_t)b * p.max_pages;
  const int share = ((older + ctas - 1) / ctas + 3) & ~3;
  const int lo = min(older, rank * share), mine = min(share, older - lo);
  auto weight_key = [&](int i) -> uint32_t {
    const int64_t at = evict_place(p, row, lo + i, hk);
    const float w = at >= 0 ? p.weights[at] : 0.f;
    return w > 0.f ? __float_as_uint(w) : 0u;   // (negative ones and NaN count as 0)
  };
  const bool held = share <= room;
  constexpr int kAhead = 8;
  if (held) {
    for (int i0 = tid; i0 < mine; i0 += kAhead * kSelectThreads) {
      // (without branches, so that all pages' numbers and then all weights are on
      // their way at once; 44 us for the call above with them)
      uint32_t k[kAhead];
      int page[kAhead];
#pragma unroll
      for (int a = 0; a < kAhead; ++a) page[a] = row[(lo + min(i0 + a * kSelectThreads, mine - 1)) >> p.ps_log2];
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const int j = lo + min(i0 + a * kSelectThreads, mine - 1);
        const bool there = page[a] >= 0 && page[a] < p.num_pages;
        const float w = p.weights[((int64_t)(there ? page[a] : 0) * p.Hk + hk) * p.page_size + (j & (p.page_size - 1))];
        k[a] = there && w > 0.f ? __float_as_uint(w) : 0u;
      }
#pragma unroll
      for (int a = 0; a < kAhead; ++a)
        if (i0 + a * kSelectThreads < mine) {
          keys[i0 + a * kSelectThreads] = k[a];
          atomicAdd(&hist[0][k[a] >> 21], 1);
        }
    }
  } else {
    for (int i = tid; i < mine; i += kSelectThreads) atomicAdd(&hist[0][weight_key(i) >> 21], 1);
  }
  auto key_of = [&](int i) -> uint32_t { return held ? keys[i] : weight_key(i); };
  // the key of the last token that stays, and how many equal to it do
  uint32_t key = 0u;
  int need = want;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t digits = pass == 2 ? 1023u : 2047u;
    if (pass > 0) {
      const int above = pass == 1 ? 21 : 10;
      for (int i = tid; i < mine; i += kSelectThreads) {
        const uint32_t k = key_of(i);
        if ((k >> above) == (key >> above)) atomicAdd(&hist[pass][(k >> shift) & digits], 1);
      }
    }
    if (ctas > 1) cluster_sync();
    else __syncthreads();
    // thread i has kMyBins digits, kBins - 1 - kMyBins i and those below, of all CTAs
    constexpr int kMyBins = kBins / kSelectThreads;
    const int at = kBins - kMyBins * (tid + 1);
    int c[kMyBins];   // (from the highest digit down)
#pragma unroll
    for (int i = 0; i < kMyBins; ++i) c[i] = 0;
    if (ctas > 1) {
      const uint32_t addr = smem_u32(&hist[pass][at]);
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r)
        if (r < ctas) {
#pragma unroll
          for (int i = 0; i < kMyBins; i += 2) {
            const int2 v = cluster_ld2(addr + 4u * i, r);
            c[kMyBins - 1 - i] += v.x;
            c[kMyBins - 2 - i] += v.y;
          }
        }
    } else {
#pragma unroll
      for (int i = 0; i < kMyBins; ++i) c[kMyBins - 1 - i] = hist[pass][at + i];
    }
    int mine_all = 0;
#pragma unroll
    for (int i = 0; i < kMyBins; ++i) mine_all += c[i];
    int2 total;
    int over = block_before(make_int2(mine_all, 0), sums, &total).x;   // counts of all higher digits
#pragma unroll
    for (int i = 0; i < kMyBins; ++i) {
      if (over < need && over + c[i] >= need) {   // (one digit of one thread)
        s_digit = at + kMyBins - 1 - i;
        s_need = need - over;
      }
      over += c[i];
    }
    __syncthreads();
    key |= (uint32_t)s_digit << shift;
    need = s_need;
    __syncthreads();
  }
  // in order: those over it, and the first `need` equal to it; a warp takes
  // neighbouring tokens, 32 at a time
  const int warp = tid >> 5, lane = tid & 31;
  const int per = ((mine + kSelectWarps - 1) / kSelectWarps + 31) & ~31;
  const int from = min(mine, warp * per), to = min(mine, from + per);
  int2 my = make_int2(0, 0);
  for (int i0 = from; i0 < to; i0 += 32) {
    const uint32_t k = i0 + lane < to ? key_of(i0 + lane) : 0u;
    my.x += __popc(__ballot_sync(0xFFFFFFFFu, i0 + lane < to && k > key));
    my.y += __popc(__ballot_sync(0xFFFFFFFFu, i0 + lane < to && k == key));
  }
  int2 total;
  int2 before = block_before(lane == 31 ? my : make_int2(0, 0), sums, &total);   // (lane 31's: of the warps before)
  if (ctas > 1) {
    if (tid == 0) counts = total;
    cluster_sync();
    for (int r = 0; r < rank; ++r) {
      const int2 v = cluster_ld2(smem_u32(&counts), r);
      before.x += v.x;
      before.y += v.y;
    }
  }
  before.x = __shfl_sync(0xFFFFFFFFu, before.x, 31);
  before.y = __shfl_sync(0xFFFFFFFFu, before.y, 31);
  for (int i0 = from; i0 < to; i0 += 32) {
    const uint32_t k = i0 + lane < to ? key_of(i0 + lane) : 0u;
    const bool over = i0 + lane < to && k > key, equal = i0 + lane < to && k == key;
    const uint32_t bo = __ballot_sync(0xFFFFFFFFu, over), be = __ballot_sync(0xFFFFFFFFu, equal), below = (1u << lane) - 1u;
    const int o = before.x + __popc(bo & below), e = before.y + __popc(be & below);
    if (over || (equal && e < need)) kept[o + min(e, need)] = lo + i0 + lane;
    before.x += __popc(bo);
    before.y += __popc(be);
  }
  if (ctas > 1) cluster_sync();   // no CTA leaves while another reads its counts
}

// A block copies `block_rows` kept rows of a (sequence, head): K, V, scales, weights.
__global__ void __launch_bounds__(kCopyThreads, 4) evict_copy_kernel(const EvictParams p, const int chunks, const int block_rows) {
  __shared__ int64_t src[kCopyThreads], dst[kCopyThreads];
  grid_dep_wait();   // the selection is complete
  grid_dep_launch();
  const int chunk = (int)(blockIdx.x % (unsigned)chunks), bh = (int)(blockIdx.x / (unsigned)chunks);
  const int b = bh / p.Hk, hk = bh % p.Hk, tid = threadIdx.x;
  const int i0 = chunk * block_rows, rows = min(block_rows, p.budget - i0);
  int64_t s = -1, d = -1;
  if (tid < rows) {
    const int i = i0 + tid, j = p.kept[(int64_t)bh * p.budget + i];
    if (j >= 0) {
      d = evict_place(p, p.new_table + (int64_t)b * p.new_pages, i, hk);
      s = evict_place(p, p.table + (int64_t)b * p.max_pages, j, hk);
    }
    src[tid] = s;
    dst[tid] = d;
  }
  if (i0 == 0 && hk == 0 && tid == 0) p.new_lens[b] = min(evict_len(p, b), p.budget);
  __syncthreads();
  // (a page outside the cache reads as zeros)
  float w = 0.f, ks = 0.f, vs = 0.f;
  const bool scales = p.scale[0] != nullptr;
  if (s >= 0) {
    w = p.weights[s];
    if (scales) {
      ks = p.scale[0][s];
      vs = p.scale[1][s];
    }
  }
  const uint32_t per = (uint32_t)p.row_bytes / 8;   // 16-byte pieces of a row's K and V together, at most 32
  const uint32_t half = per / 2, magic = (65536u + per - 1) / per;   // (x / per = x magic >> 16 for x < 2048)
  uint8_t* const k_cache = p.cache[0];
  uint8_t* const v_cache = p.cache[1];
  constexpr int kAhead = 8;
  static_assert(kCopyBytes / 16 <= 2048 && kCopyBytes / 16 <= kAhead * kCopyThreads, "a block's pieces");
  const uint32_t pieces = (uint32_t)rows * per;
  uint4 v[kAhead];
  // piece x's place from `base` (the old or the new rows), or null
  auto piece = [&](uint32_t x, const int64_t* base) -> uint8_t* {
    const uint32_t r = (x * magic) >> 16, c = x - r * per;
    const int64_t at = x < pieces ? base[r] : -1;
    return at < 0 ? nullptr : (c >= half ? v_cache + 16 * (c - half) : k_cache + 16 * c) + at * p.row_bytes;
  };
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    const uint8_t* from = piece(tid + k * kCopyThreads, src);
    v[k] = from != nullptr ? *reinterpret_cast<const uint4*>(from) : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    uint8_t* to = piece(tid + k * kCopyThreads, dst);
    if (to != nullptr) *reinterpret_cast<uint4*>(to) = v[k];
  }
  if (d >= 0) {
    p.weights[d] = w;
    if (scales) {
      p.scale[0][d] = ks;
      p.scale[1][d] = vs;
    }
  }
}

// CTAs to a (sequence, head) of at most `tokens` tokens: more while the card has room
// for them all at once (15 clusters of 8, 36 of 4, 76 of 2: a cluster lives within
// one group of SMs) and each has 2048 tokens. Eight only where four cannot hold the
// weights: adding up eight histograms costs what the smaller shares gain. (8 heads,
// d = 64, to a 64th, in clusters of 8, 4, 2 and 1: one sequence of 65536 tokens 39,
// 36, 46 and 263 us, of 16384 34, 25, 26 and 30; 16 sequences of 8192 23 in all.)
int select_cluster(long long units, long long tokens) {
  const auto most = [](int c) -> long long { return c == 8 ? 15 : c == 4 ? 36 : c == 2 ? 76 : 1ll << 40; };
  int c = tokens > 4ll * kMaxKeys ? kMaxCluster : 4;
  while (c > 1 && (units > most(c) || tokens < 2048ll * c)) c /= 2;
  return c;
}

cudaError_t launch_select(const EvictParams& p, cudaStream_t s) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static PerDeviceOnce smem_set;
  e = once_per_device(smem_set, dev, [] {
    return cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 4 * kMaxKeys);
  });
  if (e != cudaSuccess) return e;
  const long long tokens = (long long)p.max_pages * p.page_size;
  const int ctas = select_cluster((long long)p.B * p.Hk, tokens);
  const long long share = ((tokens + ctas - 1) / ctas + 3) & ~3ll;
  const int room = share < kMaxKeys ? (int)share : kMaxKeys;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.B * p.Hk * ctas));
  cfg.blockDim = dim3(kSelectThreads);
  cfg.dynamicSmemBytes = 4 * (size_t)room;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)ctas;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, evict_select_kernel, p, ctas, room);
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace

}  // namespace fa

using namespace fa;

extern "C" {

fa_status flash_attn_kv_cache_evict(void* k_cache, void* v_cache, float* k_scale, float* v_scale, float* weights,
                                    const int32_t* block_table, const int32_t* seq_lens, const int32_t* new_table,
                                    int32_t* new_lens, int32_t* kept, int B, int Hk, int d, int num_pages,
                                    int page_size, int max_pages, int new_pages, int budget, int recent,
                                    int cache_type, const fa_options* options, void* stream) {
  const bool e4m3 = cache_type == FA_CACHE_E4M3;
  if (B < 1 || Hk < 1 || num_pages < 1 || max_pages < 1 || new_pages < 1 || budget < 1 || recent < 0 || recent > budget)
    return FA_ERR_INVALID_ARG;
  if (!e4m3 && cache_type != FA_CACHE_16BIT) return FA_ERR_UNSUPPORTED;
  if (d < 8 || d > 128 || d % (e4m3 ? 16 : 8) != 0) return FA_ERR_UNSUPPORTED;
  int pl = -1;
  for (int k = 4; k <= 8; ++k)
    if (page_size == (1 << k)) pl = k;
  if (pl < 0) return FA_ERR_UNSUPPORTED;
  if ((double)max_pages * page_size > 1073741824.0 || (double)new_pages * page_size > 1073741824.0) return FA_ERR_UNSUPPORTED;
  if (budget > new_pages * page_size) return FA_ERR_INVALID_ARG;
  const int row_bytes = d * (e4m3 ? 1 : 2);
  const int fit = kCopyBytes / (2 * row_bytes), block_rows = fit < kCopyThreads ? fit : kCopyThreads;
  const int chunks = (budget + block_rows - 1) / block_rows;
  if ((double)B * Hk * chunks > 2147480000.0 || (double)B * Hk * kMaxCluster > 2147480000.0) return FA_ERR_UNSUPPORTED;
  bool f16 = false, flash_only = false;
  int st = internal_read_options(options, &f16, &flash_only);
  if (st != FA_OK) return static_cast<fa_status>(st);
  if (flash_only) return FA_ERR_UNSUPPORTED;
  const void* ptrs[] = {k_cache, v_cache, weights, block_table, seq_lens, new_table, new_lens, kept};
  for (const void* x : ptrs)
    if (x == nullptr || !aligned(x, 4)) return FA_ERR_INVALID_ARG;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16)) return FA_ERR_INVALID_ARG;
  if (e4m3 ? (k_scale == nullptr || v_scale == nullptr || !aligned(k_scale, 4) || !aligned(v_scale, 4))
           : (k_scale != nullptr || v_scale != nullptr))
    return FA_ERR_INVALID_ARG;
  unsigned int* err = nullptr;
  if ((st = internal_device_error_word(&err)) != FA_OK) return static_cast<fa_status>(st);
  EvictParams p{};
  p.cache[0] = static_cast<uint8_t*>(k_cache);
  p.cache[1] = static_cast<uint8_t*>(v_cache);
  p.scale[0] = k_scale;
  p.scale[1] = v_scale;
  p.weights = weights;
  p.table = block_table;
  p.lens = seq_lens;
  p.new_table = new_table;
  p.new_lens = new_lens;
  p.kept = kept;
  p.B = B;
  p.Hk = Hk;
  p.row_bytes = row_bytes;
  p.num_pages = num_pages;
  p.page_size = page_size;
  p.ps_log2 = pl;
  p.max_pages = max_pages;
  p.new_pages = new_pages;
  p.budget = budget;
  p.recent = recent;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (launch_select(p, s) != cudaSuccess) return FA_ERR_CUDA;
  return launch_pdl(true, evict_copy_kernel, dim3((unsigned)B * (unsigned)Hk * (unsigned)chunks), dim3(kCopyThreads), 0, s, p,
                    chunks, block_rows) == cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

}  // extern "C"
