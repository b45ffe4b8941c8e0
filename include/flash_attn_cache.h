/*
 * flash_attn_cache.h -- C ABI of serving from a paged key/value cache: the
 * writer that puts new keys and values into the cache (as 16-bit values or
 * quantised to e4m3), and the attention of the newest tokens against it.
 *
 * The method is the one of flash_attn.h: tiles of keys are streamed past
 * resident queries with an online softmax. A query of one token has no second
 * row to share a tile with, so the long axis (the keys) is what is split over
 * the GPU, and the partial results are joined by their softmax statistics.
 *
 * The cache
 * ---------
 *   k_cache, v_cache : [num_pages, Hk, page_size, d], contiguous; element type
 *       FA_CACHE_16BIT: bf16, or fp16 with options->dtype (the type of Q, K, V)
 *       FA_CACHE_E4M3:  8-bit e4m3 (4 exponent bits, 3 mantissa bits, no
 *                       infinities), with one fp32 scale per row
 *   k_scale, v_scale : fp32 [num_pages, Hk, page_size] (FA_CACHE_E4M3 only,
 *       else NULL). An element stands for payload * scale. The writer stores
 *       powers of two; the reader takes 0 and any scale from 2^-64 to 2^120
 *       (value scales of one sequence more than 2^100 apart may cost it weights
 *       below 2^-26 of the largest; one of 0 counts as 2^-64 here).
 *   page_size is 16, 32, 64, 128 or 256. Token j of a sequence lives in place
 *   j mod page_size of page block_table[b][j / page_size].
 *
 * Conventions are those of flash_attn.h (device pointers owned by the caller,
 * 16-byte aligned where not said otherwise; calls asynchronous on `stream`;
 * argument errors returned before any launch; no device memory allocated),
 * except that d is a multiple of 8 from 8 to 128 (of 16 with FA_CACHE_E4M3).
 * Of the options only dtype, wait_limit_us and test_stall are used; p_drop
 * must be 0 and tile_record NULL (FA_ERR_UNSUPPORTED otherwise). The writer
 * waits for nothing and refuses test_stall (FA_ERR_UNSUPPORTED).
 */
#ifndef FLASH_ATTN_CACHE_H
#define FLASH_ATTN_CACHE_H

#include "flash_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { FA_CACHE_16BIT = 0, FA_CACHE_E4M3 = 1 } fa_cache_type;

/*
 * Writes the keys and values of T tokens into the cache.
 *   K, V  : in, 16-bit; row (t, h) starts at element t * token_stride +
 *           h * head_stride of its tensor and holds d elements. Strides are
 *           positive multiples of 8 elements (rows may be views of a fused
 *           projection).
 *   slots : in, int64 [T] (8-byte aligned): token t goes to place
 *           slots[t] mod page_size of page slots[t] / page_size. A slot that
 *           is negative or past the cache is skipped (padding tokens). Slots
 *           that are not skipped must be distinct: of two tokens with one
 *           slot either's data, or a mix, remains.
 * Every place that no slot names is left as it was.
 * FA_CACHE_16BIT copies the rows. FA_CACHE_E4M3 stores, for each row x,
 *   scale = 2^e, e the smallest integer >= -64 with max |x| <= 448 * 2^e,
 *   payload = x / scale rounded to the nearest e4m3 value (ties to even).
 * The division is exact, so each element is rounded once: to within 2^-4 of
 * itself, or 2^-10 scale for elements below 2^-6 scale. The maximum is taken
 * over the finite elements; infinities and NaN are stored as NaN.
 *   T >= 0 (0 writes nothing), T Hk <= 2^26; 1 <= Hk <= 1024; num_pages >= 1.
 */
fa_status flash_attn_kv_cache_write(const void* K, const void* V, int64_t k_token_stride, int64_t k_head_stride,
                                    int64_t v_token_stride, int64_t v_head_stride, const int64_t* slots,
                                    int T, int Hk, int d, void* k_cache, void* v_cache, float* k_scale,
                                    float* v_scale, int num_pages, int page_size, int cache_type,
                                    const fa_options* options, void* stream);

/* Bytes of device workspace of flash_attn_cached_fwd (partial results of the
 * split keys and where each one is); 0 for an invalid shape. */
size_t flash_attn_cached_workspace_size(int B, int Nq, int Hq, int Hk, int d);

/* 0 when a call of this shape uses no workspace (few sequences that a short
 * table holds: parts are joined on chip, which is the faster way for short
 * sequences), so that it may be NULL; else 1. What counts is max_pages, since
 * the lengths are on the device. */
int flash_attn_cached_needs_workspace(int B, int Nq, int Hq, int Hk, int d, int page_size, int max_pages,
                                      int cache_type);

/*
 * Attention of the newest Nq tokens of each of B sequences (their keys and
 * values already in the cache): with n = seq_lens[b], token i of the Nq sees
 * the keys j < n - (Nq - 1 - i) of its sequence, and query head h reads
 * key/value head h / (Hq / Hk):
 *   O[b,i,h,:] = sum_j P_j V_j,  P_j = exp(S_j - LSE),
 *   LSE[b,h,i] = ln sum_j exp(S_j),  S_j = scale * Q[b,i,h,:] . K_j.
 *   Q   : in, 16-bit [B, Nq, Hq, d]; tokens (b Nq + i) are q_token_stride
 *         elements apart (a multiple of 8, at least Hq d), heads d apart
 *   O   : out, 16-bit [B, Nq, Hq, d];  LSE : out, fp32 [B, Hq, Nq]
 *   block_table : in, int32 [B, max_pages]; entries past a sequence's last
 *         page are not read. A page outside the cache reads as zeros (with
 *         FA_CACHE_E4M3 its scales too): its keys have a score of 0 and take
 *         their weight of a value of zeros.
 *   seq_lens : in, int32 [B], clamped to [0, max_pages * page_size]
 *   A token that sees no key gets O = 0, LSE = -inf. What the cache holds
 *   behind a sequence's last token does not matter (NaN neither); the keys,
 *   values and scales of the tokens before it must be finite for a finite
 *   result.
 *   B, Nq, Hk, max_pages >= 1; Hq a multiple of Hk; scale finite, positive.
 *   workspace: at least flash_attn_cached_workspace_size(B, Nq, Hq, Hk, d)
 *         bytes, 256-byte aligned; contents on entry do not matter. Calls
 *         whose kernels may overlap need workspaces of their own. May be NULL
 *         where flash_attn_cached_needs_workspace says 0.
 * 16-bit caches form P V with P rounded to 16 bits; with e4m3 the products
 * run in fp16 on exact conversions of the payloads, the scales applied to S
 * and P in fp32. Sums and statistics are fp32; results do not change from
 * call to call.
 */
fa_status flash_attn_cached_fwd(const void* Q, int64_t q_token_stride, const void* k_cache, const void* v_cache,
                                const float* k_scale, const float* v_scale, const int32_t* block_table,
                                const int32_t* seq_lens, void* O, float* LSE, int B, int Nq, int Hq, int Hk,
                                int d, int num_pages, int page_size, int max_pages, float scale, int cache_type,
                                const fa_options* options, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FLASH_ATTN_CACHE_H */
