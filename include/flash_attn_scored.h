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
 *   softcap:     0 (none), or 2^-10 to 2^10 (FA_ERR_UNSUPPORTED outside;
 *                FA_ERR_INVALID_ARG when negative or not finite). t is formed in
 *                fp32, to within 2^-21 |t| + 2^-20 softcap.
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
 * errors as there. The backward's scores must be the forward's.
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

#ifdef __cplusplus
}
#endif

#endif /* FLASH_ATTN_SCORED_H */
