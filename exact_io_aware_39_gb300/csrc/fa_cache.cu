// Serving from a paged key/value cache, for sm_103a: the writer (16-bit copy
// or quantisation to e4m3 with one scale per row), and the calls of the
// attention of the newest tokens against the cache, whose kernels are in
// fa_cached.cuh. Declarations and the contract of the calls are in
// flash_attn_cache.h and flash_attn_scored.h.
#include "fa_cached.cuh"

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

fa_status cached_fwd_call(const void* Q, int64_t q_token_stride, const void* k_cache, const void* v_cache,
                          const float* k_scale, const float* v_scale, const int32_t* block_table,
                          const int32_t* seq_lens, void* O, float* LSE, int B, int Nq, int Hq, int Hk, int d,
                          int num_pages, int page_size, int max_pages, float scale, int cache_type,
                          const fa_scores* scores, const fa_options* options, void* workspace, size_t workspace_bytes,
                          void* stream) {
  const bool e4m3 = cache_type == FA_CACHE_E4M3;
  bool f16 = false;
  CachedParams p{};
  const fa_status st = check_cached_call(Q, q_token_stride, k_cache, k_scale, block_table, seq_lens, B, Nq, Hq, Hk, d,
                                         num_pages, page_size, max_pages, scale, cache_type, scores, options, &f16, &p);
  if (st != FA_OK) return st;
  if (v_cache == nullptr || O == nullptr || LSE == nullptr || !aligned(v_cache, 16) || !aligned(O, 16) || !aligned(LSE, 4))
    return FA_ERR_INVALID_ARG;
  if (e4m3 ? (v_scale == nullptr || !aligned(v_scale, 16)) : v_scale != nullptr) return FA_ERR_INVALID_ARG;
  const CachedWorkspace w = cached_workspace_layout(B, Nq, Hq, Hk, d);
  p.cluster = cached_whole(B, Nq, Hq, Hk, d, page_size, max_pages, e4m3);
  if (!(p.cluster > 0 && workspace == nullptr) &&   // (such calls use none)
      (workspace == nullptr || !aligned(workspace, 256) || workspace_bytes < w.total))
    return FA_ERR_WORKSPACE;
  const int se = internal_device_error_word(&p.err);
  if (se != FA_OK) return static_cast<fa_status>(se);
  const int keys = cached_shape(d <= 64 ? 64 : 128, e4m3, p.cluster > 0).keys;
  CUtensorMap tk, tv, tks, tvs;
  if (!cached_maps(&tk, &tks, k_cache, k_scale, e4m3, f16, Hk, d, num_pages, page_size, keys) ||
      !cached_maps(&tv, &tvs, v_cache, v_scale, e4m3, f16, Hk, d, num_pages, page_size, keys))
    return FA_ERR_CUDA;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.o = static_cast<uint16_t*>(O);
  p.lse = LSE;
  p.part_o = reinterpret_cast<float*>(ws + w.o_off);
  p.part_ml = reinterpret_cast<float2*>(ws + w.ml_off);
  p.info = reinterpret_cast<int2*>(ws + w.info_off);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const auto launch = p.score.cap      ? launch_cached_cap
                      : p.score.slopes ? launch_cached_bias
                                       : launch_cached_score<kScorePlain>;
  const cudaError_t e = launch(e4m3, f16, tk, tv, tks, tvs, p, s);
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
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
  return cached_fwd_call(Q, q_token_stride, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, O, LSE, B, Nq, Hq, Hk,
                         d, num_pages, page_size, max_pages, scale, cache_type, nullptr, options, workspace,
                         workspace_bytes, stream);
}

fa_status flash_attn_cached_scored_fwd(const void* Q, int64_t q_token_stride, const void* k_cache, const void* v_cache,
                                       const float* k_scale, const float* v_scale, const int32_t* block_table,
                                       const int32_t* seq_lens, void* O, float* LSE, int B, int Nq, int Hq, int Hk,
                                       int d, int num_pages, int page_size, int max_pages, float scale,
                                       int cache_type, const fa_scores* scores, const fa_options* options,
                                       void* workspace, size_t workspace_bytes, void* stream) {
  return cached_fwd_call(Q, q_token_stride, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, O, LSE, B, Nq, Hq, Hk,
                         d, num_pages, page_size, max_pages, scale, cache_type, scores, options, workspace,
                         workspace_bytes, stream);
}

}  // extern "C"
