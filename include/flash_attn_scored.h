/*
 * flash_attn_scored.h -- C ABI of attention whose scores are not plain
 * products: capped by a tanh, lowered with the distance between query and key,
 * or seen past the diagonal in a prefix. The packed calls (forward and
 * backward, flash_attn_packed.h) and the cached ones (flash_attn_cache.h) take
 * such scores, and the attention that each cached token received can be added
 * up (flash_attn_cached_weights), which is what flash_attn_kv_cache_evict
 * shortens a cache by.
 *
 * The scores
 * ----------
 * With s_ij = scale * Q_i . K_j, i and j the places of query and key in their
 * sequence and h the query head,
 *   t_ij = softcap * tanh(s_ij / softcap)   (softcap 0: t_ij = s_ij),
 *   u_ij = t_ij - slopes[h] * |i - j|       (slopes NULL: u_ij = t_ij),
 * and u takes the place of s in the softmax, in LSE and in the gradients:
 *   dS_ij = P_ij (dP_ij - D_i) (1 - (t_ij / softcap)^2).
 * Causal calls with prefix_lens let every token of sequence b see its first
 * prefix_lens[b] tokens whatever the order: key j is visible to query i when
 * j <= i or j < prefix_lens[b].
 */
#ifndef FLASH_ATTN_SCORED_H
#define FLASH_ATTN_SCORED_H

#include "flash_attn_cache.h"
#include "flash_attn_packed.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 *   size:        sizeof(fa_scores), set by the caller; fields past the size a
 *                caller declares are as if 0.
 *   softcap:     0 (none), or 2^-10 to 2^10, and scale / softcap from 2^-60 to
 *                2^60 (FA_ERR_UNSUPPORTED outside; FA_ERR_INVALID_ARG when the cap
 *                is negative or not finite). t is formed in
 *                fp32, to within 2^-21 |t| + 2^-20 softcap; the gradients' factor
 *                1 - (t / softcap)^2 to within 2^-18 of itself for scores of up to
 *                12 softcaps, 2^-17 up to 21 (past them, where it is below 2^-58, it
 *                may count as 2^-60).
 *   slopes:      NULL, or fp32 [Hq] on the device (4-byte aligned), finite. They
 *                are constants of the model: no gradient of them is formed.
 *   prefix_lens: NULL, or int32 [B] on the device (4-byte aligned), clamped to
 *                [0, the sequence's length]. Needs causal = 1 (else
 *                FA_ERR_INVALID_ARG). In the cached calls it must be NULL
 *                (FA_ERR_UNSUPPORTED): what is decoded lies behind the prefix.
 * A NULL fa_scores pointer stands for plain scores.
 */
typedef struct {
  uint32_t size;
  float softcap;
  const float* slopes;
  const int32_t* prefix_lens;
} fa_scores;

/*
 * flash_attn_packed_fwd and flash_attn_packed_bwd with such scores: arguments,
 * layout, strides, workspace (flash_attn_packed_workspace_size), options and
 * errors as there. The backward's scores must be the forward's. It forms D_i as
 * the sum over j of P_ij dP_ij (where a row has few keys of weight, the rounding
 * of O would show in dQ and dK) and does not read O. (Scores without a cap, slopes
 * and prefix_lens are plain ones: the calls of flash_attn_packed.h, which read it.)
 * O is a sum in fp32 of weights of 2^14 at most: it is finite while a sequence's
 * length times its largest |V| is below 2^112, and parts of it below 2^-109 may
 * count as 0.
 */
fa_status flash_attn_packed_scored_fwd(const void* Q, const void* K, const void* V, void* O, float* LSE,
                                       const int32_t* cu_seqlens, int B, int total, int Hq, int Hk, int d,
                                       const int64_t* strides, float scale, int causal, const fa_scores* scores,
                                       const fa_options* options, void* workspace, size_t workspace_bytes,
                                       void* stream);
fa_status flash_attn_packed_scored_bwd(const void* Q, const void* K, const void* V, const void* O, const void* dO,
                                       const float* LSE, void* dQ, void* dK, void* dV, const int32_t* cu_seqlens,
                                       int B, int total, int Hq, int Hk, int d, const int64_t* strides, float scale,
                                       int causal, const fa_scores* scores, const fa_options* options,
                                       void* workspace, size_t workspace_bytes, void* stream);

/*
 * flash_attn_cached_fwd with such scores (softcap and slopes; query i of the
 * newest Nq is at place n - Nq + i of its sequence of n cached tokens, key j at
 * place j): arguments, workspace (flash_attn_cached_workspace_size,
 * flash_attn_cached_needs_workspace), options and errors as there.
 */
fa_status flash_attn_cached_scored_fwd(const void* Q, int64_t q_token_stride, const void* k_cache, const void* v_cache,
                                       const float* k_scale, const float* v_scale, const int32_t* block_table,
                                       const int32_t* seq_lens, void* O, float* LSE, int B, int Nq, int Hq, int Hk,
                                       int d, int num_pages, int page_size, int max_pages, float scale,
                                       int cache_type, const fa_scores* scores, const fa_options* options,
                                       void* workspace, size_t workspace_bytes, void* stream);

/*
 * Adds up what each cached token received from the newest Nq tokens, per
 * key/value head: for every sequence of n tokens and token j < n,
 *   weights_j = past_j + sum over i and the G query heads of exp(u_ij - LSE_i)
 * over the queries i that see key j. For the Nq newest tokens (j >= n - Nq), and
 * with past = NULL for all, past_j counts as 0: a place's former token leaves
 * nothing behind.
 *   Q, LSE  : in, as given to and by flash_attn_cached_fwd (or _scored_fwd with
 *             the same scores). Nq may be any number of newest tokens: the last
 *             32 of a prompt, for instance. A query whose LSE is -inf gives nothing.
 *   past    : in, fp32 [num_pages, Hk, page_size], or NULL
 *   weights : out, the same; may be past itself. Places of no token are left as
 *             they were, as are those of pages outside the cache.
 *   Both 8-byte aligned. A page belongs to one sequence of the call: what is left
 *   in one that two share, or that stands twice in a table, is unspecified.
 *   No workspace. Results do not change from call to call. Of the options dtype,
 *   wait_limit_us and test_stall are used, as in flash_attn_cached_fwd.
 */
fa_status flash_attn_cached_weights(const void* Q, int64_t q_token_stride, const void* k_cache, const float* k_scale,
                                    const int32_t* block_table, const int32_t* seq_lens, const float* LSE,
                                    const float* past, float* weights, int B, int Nq, int Hq, int Hk, int d,
                                    int num_pages, int page_size, int max_pages, float scale, int cache_type,
                                    const fa_scores* scores, const fa_options* options, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FLASH_ATTN_SCORED_H */
