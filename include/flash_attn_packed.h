/*
 * flash_attn_packed.h -- C ABI of exact attention, forward and backward, over
 * a packed batch: sequences of different lengths one behind another along the
 * token axis, without padding, and with grouped heads (several query heads
 * reading one key/value head). Same method, arithmetic and statistics as
 * flash_attn.h; the mask is "same sequence", and with causal "not later".
 *
 * Layout
 * ------
 *   Q, O, dO, dQ  : 16-bit [total, Hq, d];  K, V, dK, dV : 16-bit [total, Hk, d]
 *   LSE           : fp32 [Hq, total]
 *   cu_seqlens    : int32 [B + 1] on the device; sequence b is the rows
 *                   cu_seqlens[b] .. cu_seqlens[b + 1] - 1 (none when equal)
 *   strides       : host int64, for each tensor in the order of the arguments
 *                   its token stride and its head stride in elements (rows may
 *                   be views of a fused projection); NULL = contiguous. Strides
 *                   are positive multiples of 8, under 2^36; a row's d elements
 *                   are contiguous.
 * Query head h reads key/value head h / (Hq / Hk).
 *
 * Conventions are those of flash_attn.h (device pointers owned by the caller,
 * 16-byte aligned where not said otherwise; calls asynchronous on `stream`;
 * argument errors returned before any launch; no device memory allocated),
 * and:
 *  - d is a multiple of 8 from 8 to 128; a sequence has at most 131072 tokens.
 *  - Rows that belong to no sequence (behind the last one, or before the
 *    first) are not read into any result and their outputs are left as they
 *    were. What they hold does not matter (NaN neither).
 *  - Within a sequence K, V (and dO, Q in the backward pass) must be finite
 *    for finite results: a product of a zero weight and an infinity is NaN.
 *  - A sequence whose bounds decrease, leave [0, total] or span more than
 *    131072 tokens is left out, and FA_ERR_DEVICE_INTERNAL is recorded in the
 *    device error word (site 300).
 *  - Of the options dtype, wait_limit_us and test_stall are used; p_drop must
 *    be 0 and tile_record NULL (FA_ERR_UNSUPPORTED otherwise).
 *  - workspace: at least flash_attn_packed_workspace_size(...) bytes, 256-byte
 *    aligned; contents on entry do not matter. Calls whose kernels may overlap
 *    need workspaces of their own. A forward call of at most 128 sequences uses
 *    none (workspace may be NULL).
 *  - Launches are sized by B and total, since the bounds are on the device:
 *    tensors much longer than their sequences cost time for rows that no
 *    sequence has.
 */
#ifndef FLASH_ATTN_PACKED_H
#define FLASH_ATTN_PACKED_H

#include "flash_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of device workspace of a forward (backward = 0) or backward (1) call:
 * the list of work items and, for the backward, the fp32 dQ accumulator and
 * two row vectors, over sequences padded to multiples of 128 tokens (at most
 * total + 128 B of them), and, where the call's key tiles alone would not fill
 * the GPU, up to 16 fp32 parts of dK and dV. 0 for an invalid shape. */
size_t flash_attn_packed_workspace_size(int B, int total, int Hq, int Hk, int d, int backward);

/*
 * Forward pass. For every sequence, head h and token i of it,
 *   O[i,h,:] = sum_j P_ij V[j,h',:],  P_ij = exp(S_ij - LSE[h,i]),
 *   LSE[h,i] = ln sum_j exp(S_ij),    S_ij = scale * Q[i,h,:] . K[j,h',:]
 * over the tokens j of the sequence (causal: j <= i), h' = h / (Hq / Hk).
 *   strides: 8 values (Q, K, V, O).  B, total >= 0 (0: nothing to do);
 *   Hq a multiple of Hk >= 1; scale finite and positive; causal 0 or 1.
 */
fa_status flash_attn_packed_fwd(const void* Q, const void* K, const void* V, void* O, float* LSE,
                                const int32_t* cu_seqlens, int B, int total, int Hq, int Hk, int d,
                                const int64_t* strides, float scale, int causal, const fa_options* options,
                                void* workspace, size_t workspace_bytes, void* stream);

/*
 * Backward pass by recomputation, from the forward's inputs and outputs and
 * the output gradient dO (formulas as in flash_attn_bwd; dK and dV of a
 * key/value head are summed over its query heads in fp32, in a fixed order).
 * The fp32 partial sums of dQ are added in the order they become ready, so
 * dQ may differ in its last bits from call to call; dK and dV do not.
 *   strides: 16 values (Q, K, V, O, dO, dQ, dK, dV).
 */
fa_status flash_attn_packed_bwd(const void* Q, const void* K, const void* V, const void* O, const void* dO,
                                const float* LSE, void* dQ, void* dK, void* dV, const int32_t* cu_seqlens,
                                int B, int total, int Hq, int Hk, int d, const int64_t* strides, float scale,
                                int causal, const fa_options* options, void* workspace, size_t workspace_bytes,
                                void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FLASH_ATTN_PACKED_H */
