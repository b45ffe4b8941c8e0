// A paged cache shortened to the tokens with the most accumulated attention
// (flash_attn_kv_cache_evict in flash_attn_cache.h), for sm_103a, in two kernels:
// one finds the tokens that stay, for each sequence and key/value head by itself,
// the other copies their rows to the pages of the new table.
//
// The selection: a weight >= 0 orders as its bits do, so the weight of the last
// token that stays is found from the top, eight bits at a time (a histogram of
// the tokens that agree with what is known so far, summed from above), and a pass
// over the tokens in order then lists those over it and as many of those equal to
// it as are missing, the first ones. Bound: the weights are read from L2 five
// times; a few us a pass for 65536 tokens.
//
// The copy is bound by memory: it reads and writes each kept row once.
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

constexpr int kSelectThreads = 1024;
constexpr int kCopyThreads = 256, kCopyRows = 64;

__device__ __forceinline__ int evict_len(const EvictParams& p, int b) {
  const int n = p.lens[b], cap = p.max_pages << p.ps_log2;
  return n < 0 ? 0 : (n > cap ? cap : n);
}

// Place of token j of head hk in a table's pages ([num_pages, Hk, page_size]), or -1.
__device__ __forceinline__ int64_t evict_place(const EvictParams& p, const int32_t* row, int j, int hk) {
  const int page = row[j >> p.ps_log2];
  return page >= 0 && page < p.num_pages ? ((int64_t)page * p.Hk + hk) * p.page_size + (j & (p.page_size - 1)) : -1;
}

// A block per (sequence, head).
__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(const EvictParams p) {
  __shared__ int hist[256], warp_sum[2][32];
  __shared__ uint32_t s_key;
  __shared__ int s_need;
  grid_dep_wait();
  grid_dep_launch();
  const int b = (int)blockIdx.x / p.Hk, hk = (int)blockIdx.x % p.Hk;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = evict_len(p, b);
  int32_t* kept = p.kept + (int64_t)blockIdx.x * p.budget;
  if (n <= p.budget) {
    for (int j = tid; j < p.budget; j += kSelectThreads) kept[j] = j < n ? j : -1;
    return;
  }
  const int32_t* row = p.table + (int64_t)b * p.max_pages;
  const int older = n - p.recent, want = p.budget - p.recent;   // 0 <= want < older
  for (int i = tid; i < p.recent; i += kSelectThreads) kept[want + i] = older + i;
  if (want == 0) return;
  auto key_of = [&](int j) -> uint32_t {
    const int64_t at = evict_place(p, row, j, hk);
    const float w = at >= 0 ? p.weights[at] : 0.f;
    return w > 0.f ? __float_as_uint(w) : 0u;   // (negative ones and NaN count as 0)
  };
  // the key of the last token that stays, and how many equal to it do
  uint32_t key = 0u;
  int need = want;
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    for (int j = tid; j < older; j += kSelectThreads) {
      const uint32_t k = key_of(j);
      if (shift == 24 || (k >> (shift + 8)) == (key >> (shift + 8))) atomicAdd(&hist[(k >> shift) & 255u], 1);
    }
    __syncthreads();
    if (warp == 0) {
      // lane l has digits 255 - 8 l and the seven below it
      int c[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += c[i] = hist[255 - 8 * lane - i];
      int upto = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, upto, o);
        if (lane >= o) upto += y;
      }
      int above = upto - sum;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (above < need && above + c[i] >= need) {   // (one digit of one lane)
          s_key = key | ((uint32_t)(255 - 8 * lane - i) << shift);
          s_need = need - above;
        }
        above += c[i];
      }
    }
    __syncthreads();
    key = s_key;
    need = s_need;
  }
  // in order: those over it, and the first `need` equal to it
  int over = 0, equal = 0;   // among the tokens before this round's
  for (int base = 0, round = 0; base < older; base += kSelectThreads, round ^= 1) {
    const int j = base + tid;
    const uint32_t k = j < older ? key_of(j) : 0u;
    const bool gt = j < older && k > key, eq = j < older && k == key;
    const uint32_t bg = __ballot_sync(0xFFFFFFFFu, gt), be = __ballot_sync(0xFFFFFFFFu, eq);
    if (lane == 0) warp_sum[round][warp] = __popc(bg) | (__popc(be) << 16);
    __syncthreads();
    int x = warp_sum[round][lane];   // counts of at most 1024 in each half
    int upto = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += y;
    }
    const int all = __shfl_sync(0xFFFFFFFFu, upto, 31);
    const int mine = __shfl_sync(0xFFFFFFFFu, upto - x, warp);
    const uint32_t below = (1u << lane) - 1u;
    const int g0 = over + (mine & 0xFFFF) + __popc(bg & below), e0 = equal + (mine >> 16) + __popc(be & below);
    if (gt || (eq && e0 < need)) kept[g0 + min(e0, need)] = j;
    over += all & 0xFFFF;
    equal += all >> 16;
  }
}

// A block copies kCopyRows kept rows of a (sequence, head): K, V, scales, weights.
__global__ void __launch_bounds__(kCopyThreads) evict_copy_kernel(const EvictParams p, int chunks) {
  __shared__ int64_t src[kCopyRows], dst[kCopyRows];
  grid_dep_wait();   // the selection is complete
  grid_dep_launch();
  const int chunk = (int)(blockIdx.x % (unsigned)chunks), bh = (int)(blockIdx.x / (unsigned)chunks);
  const int b = bh / p.Hk, hk = bh % p.Hk, tid = threadIdx.x;
  const int i0 = chunk * kCopyRows, rows = min(kCopyRows, p.budget - i0);
  if (tid < rows) {
    const int i = i0 + tid, j = p.kept[(int64_t)bh * p.budget + i];
    int64_t s = -1, d = -1;
    if (j >= 0) {
      d = evict_place(p, p.new_table + (int64_t)b * p.new_pages, i, hk);
      s = evict_place(p, p.table + (int64_t)b * p.max_pages, j, hk);
      if (d >= 0) {
        // (a page outside the cache reads as zeros)
        p.weights[d] = s >= 0 ? p.weights[s] : 0.f;
        if (p.scale[0] != nullptr) {
          p.scale[0][d] = s >= 0 ? p.scale[0][s] : 0.f;
          p.scale[1][d] = s >= 0 ? p.scale[1][s] : 0.f;
        }
      }
    }
    src[tid] = s;
    dst[tid] = d;
  }
  if (i0 == 0 && hk == 0 && tid == 0) p.new_lens[b] = min(evict_len(p, b), p.budget);
  __syncthreads();
  const int per = p.row_bytes / 8;   // 16-byte pieces of a row's K and V together
  const int half = per / 2;
  constexpr int kAhead = 8;
  for (int x0 = tid; x0 < rows * per; x0 += kAhead * kCopyThreads) {
    uint4 v[kAhead];
    uint8_t* to[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int x = x0 + k * kCopyThreads;
      to[k] = nullptr;
      if (x < rows * per) {
        const int r = x / per, c = x % per;
        const int side = c >= half ? 1 : 0, off = 16 * (c - side * half);
        if (dst[r] >= 0) to[k] = p.cache[side] + dst[r] * p.row_bytes + off;
        v[k] = dst[r] >= 0 && src[r] >= 0 ? *reinterpret_cast<const uint4*>(p.cache[side] + src[r] * p.row_bytes + off)
                                          : make_uint4(0u, 0u, 0u, 0u);
      }
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (to[k] != nullptr) *reinterpret_cast<uint4*>(to[k]) = v[k];
  }
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
  const int chunks = (budget + kCopyRows - 1) / kCopyRows;
  if ((double)B * Hk * chunks > 2147480000.0) return FA_ERR_UNSUPPORTED;
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
  p.row_bytes = d * (e4m3 ? 1 : 2);
  p.num_pages = num_pages;
  p.page_size = page_size;
  p.ps_log2 = pl;
  p.max_pages = max_pages;
  p.new_pages = new_pages;
  p.budget = budget;
  p.recent = recent;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (launch_pdl(true, evict_select_kernel, dim3((unsigned)(B * Hk)), dim3(kSelectThreads), 0, s, p) != cudaSuccess)
    return FA_ERR_CUDA;
  return launch_pdl(true, evict_copy_kernel, dim3((unsigned)B * (unsigned)Hk * (unsigned)chunks), dim3(kCopyThreads), 0, s, p,
                    chunks) == cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

}  // extern "C"
