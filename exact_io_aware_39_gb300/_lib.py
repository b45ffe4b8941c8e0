"""ctypes binding of libflashattn.so: the C ABI of include/flash_attn.h,
flash_attn_packed.h, flash_attn_cache.h, flash_attn_scored.h and standard_attn.h under the same names,
plus thin helpers that take torch tensors.

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI. There is no CPU or PyTorch fallback; if the shared
library is missing or does not load, every call raises.
"""
from __future__ import annotations

import ctypes
import os
import struct

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libflashattn.so")

FA_OK = 0
STATUS_NAMES = {
    0: "FA_OK", 1: "FA_ERR_INVALID_ARG", 2: "FA_ERR_UNSUPPORTED", 3: "FA_ERR_WORKSPACE",
    4: "FA_ERR_CUDA", 5: "FA_ERR_DEVICE_TIMEOUT", 6: "FA_ERR_DEVICE_INTERNAL",
    7: "FA_ERR_SCRATCH_LIMIT",
}
FA_ERR_SCRATCH_LIMIT = 7
BWD_NOALLOC_SCRATCH_BYTES = 64 << 20

# every symbol the headers in include/ declare
EXPORTS = [
    "flash_attn_fwd", "flash_attn_fwd_ex", "flash_attn_bwd_workspace_size", "flash_attn_bwd",
    "flash_attn_bwd_ex", "flash_attn_bwd_noalloc",
    "flash_attn_tile_map",
    "flash_attn_get_device_error", "flash_attn_set_profile_events", "flash_attn_status_string",
    "flash_attn_version",
    "flash_attn_packed_workspace_size", "flash_attn_packed_fwd", "flash_attn_packed_bwd",
    "flash_attn_kv_cache_write", "flash_attn_cached_workspace_size", "flash_attn_cached_needs_workspace",
    "flash_attn_cached_fwd",
    "flash_attn_packed_scored_fwd", "flash_attn_packed_scored_bwd", "flash_attn_cached_scored_fwd",
    "flash_attn_cached_weights", "flash_attn_kv_cache_evict",
    "standard_attn_workspace_size", "standard_attn_fwd", "standard_attn_bwd",
]


FA_DTYPE_BF16, FA_DTYPE_F16 = 0, 1


class fa_options(ctypes.Structure):
    """Mirror of the C struct fa_options (size is set by the constructor)."""
    _fields_ = [("size", ctypes.c_uint32), ("dtype", ctypes.c_int32), ("p_drop", ctypes.c_float),
                ("reserved", ctypes.c_uint32), ("seed", ctypes.c_uint64),
                ("tile_record", ctypes.c_void_p), ("wait_limit_us", ctypes.c_uint32),
                ("test_stall", ctypes.c_uint32)]

    def __init__(self, dtype=FA_DTYPE_BF16, p_drop=0.0, seed=0, tile_record=None, wait_limit_us=0,
                 test_stall=0):
        super().__init__(ctypes.sizeof(fa_options), dtype, float(p_drop), 0, int(seed), tile_record,
                         int(wait_limit_us), int(test_stall))


class fa_scores(ctypes.Structure):
    """Mirror of the C struct fa_scores (size is set by the constructor)."""
    _fields_ = [("size", ctypes.c_uint32), ("softcap", ctypes.c_float), ("slopes", ctypes.c_void_p),
                ("prefix_lens", ctypes.c_void_p)]

    def __init__(self, softcap=0.0, slopes=None, prefix_lens=None):
        super().__init__(ctypes.sizeof(fa_scores), float(softcap), slopes, prefix_lens)


class FlashAttnError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}")


_lib = None


def load(path=LIB_PATH):
    """Loads (once) and returns the ctypes handle of the library."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m exact_io_aware_39_gb300.build`")
    lib = ctypes.CDLL(path)
    vp, i32, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.flash_attn_fwd.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, f32, i32, vp, vp, vp]
    lib.flash_attn_fwd.restype = i32
    opt_p = ctypes.POINTER(fa_options)
    lib.flash_attn_fwd_ex.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, f32, i32, vp, vp, opt_p, vp]
    lib.flash_attn_fwd_ex.restype = i32
    lib.flash_attn_bwd_ex.argtypes = [vp] * 9 + [i32, i32, i32, i32, f32, i32, vp, vp, opt_p, vp, sz, vp]
    lib.flash_attn_bwd_ex.restype = i32
    lib.flash_attn_bwd_workspace_size.argtypes = [i32, i32, i32, i32]
    lib.flash_attn_bwd_workspace_size.restype = sz
    lib.flash_attn_bwd.argtypes = [vp] * 9 + [i32, i32, i32, i32, f32, i32, vp, vp, vp, sz, vp]
    lib.flash_attn_bwd.restype = i32
    lib.flash_attn_bwd_noalloc.argtypes = [vp] * 9 + [i32, i32, i32, i32, f32, i32, vp, vp, vp]
    lib.flash_attn_bwd_noalloc.restype = i32
    lib.flash_attn_tile_map.argtypes = [i32, i32, i32, vp, vp, vp, vp]
    lib.flash_attn_tile_map.restype = i32
    lib.flash_attn_get_device_error.argtypes = [ctypes.POINTER(ctypes.c_uint32)]
    lib.flash_attn_get_device_error.restype = i32
    lib.flash_attn_set_profile_events.argtypes = [vp, vp]
    lib.flash_attn_set_profile_events.restype = i32
    lib.flash_attn_status_string.argtypes = [i32]
    lib.flash_attn_status_string.restype = ctypes.c_char_p
    lib.flash_attn_version.argtypes = []
    lib.flash_attn_version.restype = i32
    i64 = ctypes.c_int64
    lib.flash_attn_packed_workspace_size.argtypes = [i32] * 6
    lib.flash_attn_packed_workspace_size.restype = sz
    lib.flash_attn_packed_fwd.argtypes = [vp] * 6 + [i32] * 5 + [vp, f32, i32, opt_p, vp, sz, vp]
    lib.flash_attn_packed_fwd.restype = i32
    lib.flash_attn_packed_bwd.argtypes = [vp] * 10 + [i32] * 5 + [vp, f32, i32, opt_p, vp, sz, vp]
    lib.flash_attn_packed_bwd.restype = i32
    # (scores: an fa_scores by reference, or its bytes)
    lib.flash_attn_packed_scored_fwd.argtypes = [vp] * 6 + [i32] * 5 + [vp, f32, i32, vp, opt_p, vp, sz, vp]
    lib.flash_attn_packed_scored_fwd.restype = i32
    lib.flash_attn_packed_scored_bwd.argtypes = [vp] * 10 + [i32] * 5 + [vp, f32, i32, vp, opt_p, vp, sz, vp]
    lib.flash_attn_packed_scored_bwd.restype = i32
    lib.flash_attn_kv_cache_write.argtypes = [vp, vp, i64, i64, i64, i64, vp, i32, i32, i32, vp, vp, vp, vp, i32, i32,
                                              i32, opt_p, vp]
    lib.flash_attn_kv_cache_write.restype = i32
    lib.flash_attn_cached_workspace_size.argtypes = [i32] * 5
    lib.flash_attn_cached_workspace_size.restype = sz
    lib.flash_attn_cached_needs_workspace.argtypes = [i32] * 8
    lib.flash_attn_cached_needs_workspace.restype = i32
    lib.flash_attn_cached_fwd.argtypes = [vp, i64] + [vp] * 8 + [i32] * 8 + [f32, i32, opt_p, vp, sz, vp]
    lib.flash_attn_cached_fwd.restype = i32
    lib.flash_attn_cached_scored_fwd.argtypes = [vp, i64] + [vp] * 8 + [i32] * 8 + [f32, i32, vp, opt_p, vp, sz, vp]
    lib.flash_attn_cached_scored_fwd.restype = i32
    lib.flash_attn_cached_weights.argtypes = [vp, i64] + [vp] * 7 + [i32] * 8 + [f32, i32, vp, opt_p, vp]
    lib.flash_attn_cached_weights.restype = i32
    lib.flash_attn_kv_cache_evict.argtypes = [vp] * 10 + [i32] * 10 + [opt_p, vp]
    lib.flash_attn_kv_cache_evict.restype = i32
    lib.standard_attn_workspace_size.argtypes = [i32, i32, i32]
    lib.standard_attn_workspace_size.restype = sz
    lib.standard_attn_fwd.argtypes = [vp] * 5 + [i32, i32, i32, i32, f32, i32, vp, vp, opt_p, i32, vp, sz, vp]
    lib.standard_attn_fwd.restype = i32
    lib.standard_attn_bwd.argtypes = [vp] * 7 + [i32, i32, i32, i32, f32, opt_p, i32, vp, sz, vp]
    lib.standard_attn_bwd.restype = i32
    _lib = lib
    return lib


# ---------------------------------------------------------------------------
# raw C-ABI calls (same names and argument order as the header)
# ---------------------------------------------------------------------------

def flash_attn_fwd(Q, K, V, O, LSE, B, H, N, d, scale, causal, kv_len, block_mask, stream):
    return load().flash_attn_fwd(Q, K, V, O, LSE, B, H, N, d, scale, causal, kv_len, block_mask, stream)


def flash_attn_fwd_ex(Q, K, V, O, LSE, B, H, N, d, scale, causal, kv_len, block_mask, options, stream):
    return load().flash_attn_fwd_ex(Q, K, V, O, LSE, B, H, N, d, scale, causal, kv_len, block_mask,
                                    None if options is None else ctypes.byref(options), stream)


def flash_attn_bwd_ex(Q, K, V, O, dO, LSE, dQ, dK, dV, B, H, N, d, scale, causal, kv_len, block_mask,
                      options, workspace, workspace_bytes, stream):
    return load().flash_attn_bwd_ex(Q, K, V, O, dO, LSE, dQ, dK, dV, B, H, N, d, scale, causal, kv_len,
                                    block_mask, None if options is None else ctypes.byref(options),
                                    workspace, workspace_bytes, stream)


def flash_attn_bwd_workspace_size(B, H, N, d):
    return load().flash_attn_bwd_workspace_size(B, H, N, d)


def flash_attn_bwd(Q, K, V, O, dO, LSE, dQ, dK, dV, B, H, N, d, scale, causal, kv_len, block_mask,
                   workspace, workspace_bytes, stream):
    return load().flash_attn_bwd(Q, K, V, O, dO, LSE, dQ, dK, dV, B, H, N, d, scale, causal, kv_len,
                                 block_mask, workspace, workspace_bytes, stream)


def flash_attn_bwd_noalloc(Q, K, V, O, dO, LSE, dQ, dK, dV, B, H, N, d, scale, causal, kv_len,
                           block_mask, stream):
    """Backward without a workspace argument: for callers that cannot allocate
    device memory (see the header); scratch comes from a fixed 64 MiB array."""
    return load().flash_attn_bwd_noalloc(Q, K, V, O, dO, LSE, dQ, dK, dV, B, H, N, d, scale, causal,
                                         kv_len, block_mask, stream)


def flash_attn_tile_map(B, N, causal, kv_len, block_mask, out, stream):
    return load().flash_attn_tile_map(B, N, causal, kv_len, block_mask, out, stream)


def flash_attn_get_device_error():
    detail = (ctypes.c_uint32 * 4)()
    st = load().flash_attn_get_device_error(detail)
    return st, list(detail)


def flash_attn_set_profile_events(start_event, stop_event):
    return load().flash_attn_set_profile_events(start_event, stop_event)


def flash_attn_status_string(status):
    return load().flash_attn_status_string(status).decode()


def flash_attn_version():
    return load().flash_attn_version()


def flash_attn_packed_workspace_size(B, total, Hq, Hk, d, backward):
    return load().flash_attn_packed_workspace_size(B, total, Hq, Hk, d, backward)


def flash_attn_packed_fwd(Q, K, V, O, LSE, cu_seqlens, B, total, Hq, Hk, d, strides, scale, causal, options, workspace,
                          workspace_bytes, stream):
    return load().flash_attn_packed_fwd(Q, K, V, O, LSE, cu_seqlens, B, total, Hq, Hk, d, strides, scale, causal,
                                        None if options is None else ctypes.byref(options), workspace,
                                        workspace_bytes, stream)


def flash_attn_packed_bwd(Q, K, V, O, dO, LSE, dQ, dK, dV, cu_seqlens, B, total, Hq, Hk, d, strides, scale, causal,
                          options, workspace, workspace_bytes, stream):
    return load().flash_attn_packed_bwd(Q, K, V, O, dO, LSE, dQ, dK, dV, cu_seqlens, B, total, Hq, Hk, d, strides, scale,
                                        causal, None if options is None else ctypes.byref(options), workspace,
                                        workspace_bytes, stream)


def flash_attn_packed_scored_fwd(Q, K, V, O, LSE, cu_seqlens, B, total, Hq, Hk, d, strides, scale, causal, scores, options,
                                 workspace, workspace_bytes, stream):
    return load().flash_attn_packed_scored_fwd(Q, K, V, O, LSE, cu_seqlens, B, total, Hq, Hk, d, strides, scale, causal,
                                               None if scores is None else ctypes.byref(scores),
                                               None if options is None else ctypes.byref(options), workspace,
                                               workspace_bytes, stream)


def flash_attn_packed_scored_bwd(Q, K, V, O, dO, LSE, dQ, dK, dV, cu_seqlens, B, total, Hq, Hk, d, strides, scale,
                                 causal, scores, options, workspace, workspace_bytes, stream):
    return load().flash_attn_packed_scored_bwd(Q, K, V, O, dO, LSE, dQ, dK, dV, cu_seqlens, B, total, Hq, Hk, d,
                                               strides, scale, causal,
                                               None if scores is None else ctypes.byref(scores),
                                               None if options is None else ctypes.byref(options), workspace,
                                               workspace_bytes, stream)


def flash_attn_kv_cache_write(K, V, k_token_stride, k_head_stride, v_token_stride, v_head_stride, slots, T, Hk, d,
                              k_cache, v_cache, k_scale, v_scale, num_pages, page_size, cache_type, options, stream):
    return load().flash_attn_kv_cache_write(K, V, k_token_stride, k_head_stride, v_token_stride, v_head_stride, slots,
                                            T, Hk, d, k_cache, v_cache, k_scale, v_scale, num_pages, page_size,
                                            cache_type, None if options is None else ctypes.byref(options), stream)


def flash_attn_cached_workspace_size(B, Nq, Hq, Hk, d):
    return load().flash_attn_cached_workspace_size(B, Nq, Hq, Hk, d)


def flash_attn_cached_needs_workspace(B, Nq, Hq, Hk, d, page_size, max_pages, cache_type):
    return load().flash_attn_cached_needs_workspace(B, Nq, Hq, Hk, d, page_size, max_pages, cache_type)


def flash_attn_cached_fwd(Q, q_token_stride, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, O, LSE, B, Nq,
                          Hq, Hk, d, num_pages, page_size, max_pages, scale, cache_type, options, workspace,
                          workspace_bytes, stream):
    return load().flash_attn_cached_fwd(Q, q_token_stride, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, O,
                                        LSE, B, Nq, Hq, Hk, d, num_pages, page_size, max_pages, scale, cache_type,
                                        None if options is None else ctypes.byref(options), workspace,
                                        workspace_bytes, stream)


def flash_attn_cached_scored_fwd(Q, q_token_stride, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, O, LSE, B,
                                 Nq, Hq, Hk, d, num_pages, page_size, max_pages, scale, cache_type, scores, options,
                                 workspace, workspace_bytes, stream):
    return load().flash_attn_cached_scored_fwd(Q, q_token_stride, k_cache, v_cache, k_scale, v_scale, block_table,
                                               seq_lens, O, LSE, B, Nq, Hq, Hk, d, num_pages, page_size, max_pages,
                                               scale, cache_type, None if scores is None else ctypes.byref(scores),
                                               None if options is None else ctypes.byref(options), workspace,
                                               workspace_bytes, stream)


def flash_attn_cached_weights(Q, q_token_stride, k_cache, k_scale, block_table, seq_lens, LSE, past, weights, B, Nq, Hq,
                              Hk, d, num_pages, page_size, max_pages, scale, cache_type, scores, options, stream):
    return load().flash_attn_cached_weights(Q, q_token_stride, k_cache, k_scale, block_table, seq_lens, LSE, past,
                                            weights, B, Nq, Hq, Hk, d, num_pages, page_size, max_pages, scale,
                                            cache_type, None if scores is None else ctypes.byref(scores),
                                            None if options is None else ctypes.byref(options), stream)


def flash_attn_kv_cache_evict(k_cache, v_cache, k_scale, v_scale, weights, block_table, seq_lens, new_table, new_lens,
                              kept, B, Hk, d, num_pages, page_size, max_pages, new_pages, budget, recent, cache_type,
                              options, stream):
    return load().flash_attn_kv_cache_evict(k_cache, v_cache, k_scale, v_scale, weights, block_table, seq_lens,
                                            new_table, new_lens, kept, B, Hk, d, num_pages, page_size, max_pages,
                                            new_pages, budget, recent, cache_type,
                                            None if options is None else ctypes.byref(options), stream)


def standard_attn_workspace_size(B, H, N):
    return load().standard_attn_workspace_size(B, H, N)


STANDARD_ATTN_S16 = 1


def standard_attn_fwd(Q, K, V, O, LSE, B, H, N, d, scale, causal, kv_len, block_mask, options, flags, workspace,
                      workspace_bytes, stream):
    return load().standard_attn_fwd(Q, K, V, O, LSE, B, H, N, d, scale, causal, kv_len, block_mask,
                                    None if options is None else ctypes.byref(options), flags, workspace,
                                    workspace_bytes, stream)


def standard_attn_bwd(Q, K, V, dO, dQ, dK, dV, B, H, N, d, scale, options, flags, workspace, workspace_bytes,
                      stream):
    return load().standard_attn_bwd(Q, K, V, dO, dQ, dK, dV, B, H, N, d, scale,
                                    None if options is None else ctypes.byref(options), flags, workspace,
                                    workspace_bytes, stream)


# ---------------------------------------------------------------------------
# torch helpers (device memory and streams come from PyTorch)
# ---------------------------------------------------------------------------

def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(st, where):
    if st != FA_OK:
        raise FlashAttnError(st, where)


def _check_inputs(*ts):
    """Validates the tensors and returns the fa_options for their dtype."""
    import torch
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("tensors must be contiguous CUDA tensors")
    dt = ts[0].dtype
    if dt not in (torch.bfloat16, torch.float16):
        raise ValueError("Q, K, V must be bfloat16 or float16 [B, H, N, d]")
    for t in ts:
        if t is not None and (t.dtype != dt or t.dim() != 4):
            raise ValueError("Q, K, V (and O, dO) must share one 16-bit dtype and be [B, H, N, d]")
    return fa_options(FA_DTYPE_F16 if dt == torch.float16 else FA_DTYPE_BF16)


def _mask_args(kv_len, block_mask):
    import torch
    if kv_len is not None and (kv_len.dtype != torch.int32 or not kv_len.is_cuda):
        raise ValueError("kv_len must be a CUDA int32 tensor [B]")
    if block_mask is not None and (block_mask.dtype != torch.uint8 or not block_mask.is_cuda):
        raise ValueError("block_mask must be a CUDA uint8 tensor [nT, nT]")
    return _ptr(kv_len), _ptr(block_mask)


def _set_checks(opts, tile_record, wait_limit_us, test_stall):
    """Fills the checking fields of fa_options: tile_record (a zeroed CUDA
    uint8 tensor [B, H, nT, nT] or None), wait_limit_us, test_stall."""
    import torch
    if tile_record is not None:
        if tile_record.dtype != torch.uint8 or not tile_record.is_cuda or not tile_record.is_contiguous():
            raise ValueError("tile_record must be a contiguous CUDA uint8 tensor [B, H, nT, nT]")
        opts.tile_record = tile_record.data_ptr()
    opts.wait_limit_us = int(wait_limit_us)
    opts.test_stall = int(test_stall)


def attention_fwd(q, k, v, scale, causal=False, kv_len=None, block_mask=None, out=None, lse=None,
                  stream=None, p_drop=0.0, seed=0, tile_record=None, wait_limit_us=0, test_stall=0):
    """O, LSE = attention(q, k, v) on the GPU. q, k, v: bf16 or fp16 [B, H, N, d];
    p_drop > 0 applies dropout to P (mask from Philox4x32-10 keyed by seed).
    tile_record, wait_limit_us and test_stall are the checking options of
    fa_options (see include/flash_attn.h)."""
    import torch
    opts = _check_inputs(q, k, v)
    opts.p_drop, opts.seed = float(p_drop), int(seed)
    _set_checks(opts, tile_record, wait_limit_us, test_stall)
    B, H, N, d = q.shape
    o = torch.empty_like(q) if out is None else out
    l = torch.empty((B, H, N), dtype=torch.float32, device=q.device) if lse is None else lse
    kv_p, bm_p = _mask_args(kv_len, block_mask)
    st = flash_attn_fwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(l), B, H, N, d, float(scale),
                           int(bool(causal)), kv_p, bm_p, opts, _stream(stream))
    _check(st, "flash_attn_fwd_ex")
    return o, l


def attention_bwd(q, k, v, o, do, lse, scale, causal=False, kv_len=None, block_mask=None,
                  workspace=None, dq=None, dk=None, dv=None, stream=None, p_drop=0.0, seed=0,
                  tile_record=None, wait_limit_us=0, test_stall=0):
    """dQ, dK, dV of attention on the GPU (recomputing S, P and the dropout
    mask on chip); p_drop and seed must match the forward call."""
    import torch
    opts = _check_inputs(q, k, v, o, do)
    opts.p_drop, opts.seed = float(p_drop), int(seed)
    _set_checks(opts, tile_record, wait_limit_us, test_stall)
    B, H, N, d = q.shape
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    need = flash_attn_bwd_workspace_size(B, H, N, d)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    kv_p, bm_p = _mask_args(kv_len, block_mask)
    st = flash_attn_bwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(dq), _ptr(dk),
                           _ptr(dv), B, H, N, d, float(scale), int(bool(causal)), kv_p, bm_p, opts,
                           _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "flash_attn_bwd_ex")
    return dq, dk, dv


def tile_map(B, N, causal=False, kv_len=None, block_mask=None, device="cuda", stream=None):
    """uint8 [B, nT, nT] tile states the kernels use (0 skip, 1 full, 2 partial)."""
    import torch
    nT = (N + 127) // 128
    out = torch.empty((B, nT, nT), dtype=torch.uint8, device=device)
    kv_p, bm_p = _mask_args(kv_len, block_mask)
    st = flash_attn_tile_map(B, N, int(bool(causal)), kv_p, bm_p, _ptr(out), _stream(stream))
    _check(st, "flash_attn_tile_map")
    return out


def profile_next_call(start, stop):
    """Record torch.cuda.Event start/stop around the dominant kernel of the
    next attention_fwd/attention_bwd call of this thread."""
    st = flash_attn_set_profile_events(ctypes.c_void_p(start.cuda_event), ctypes.c_void_p(stop.cuda_event))
    _check(st, "flash_attn_set_profile_events")


def device_error():
    """(status, [code, site, block, thread]) of the device error word; clears it."""
    return flash_attn_get_device_error()


def standard_attention_fwd(q, k, v, scale, causal=False, kv_len=None, block_mask=None, workspace=None,
                           stream=None, s16=False):
    """Standard (materialising) attention on the GPU: (O, LSE, workspace); the
    workspace holds S and P and must be passed to standard_attention_bwd.
    s16=True stores S (and later dP) in the 16-bit input type."""
    import torch
    opts = _check_inputs(q, k, v)
    B, H, N, d = q.shape
    o = torch.empty_like(q)
    l = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    need = standard_attn_workspace_size(B, H, N)
    if need == 0:
        raise FlashAttnError(2, "standard_attn_workspace_size")
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    kv_p, bm_p = _mask_args(kv_len, block_mask)
    st = standard_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(l), B, H, N, d, float(scale),
                           int(bool(causal)), kv_p, bm_p, opts, STANDARD_ATTN_S16 if s16 else 0, _ptr(workspace),
                           workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "standard_attn_fwd")
    return o, l, workspace


def standard_attention_bwd(q, k, v, do, workspace, scale, stream=None, s16=False):
    """dQ, dK, dV of standard attention from the P the forward call stored
    (s16 as in the forward call)."""
    import torch
    opts = _check_inputs(q, k, v, do)
    B, H, N, d = q.shape
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    st = standard_attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(do), _ptr(dq), _ptr(dk), _ptr(dv), B, H, N, d,
                           float(scale), opts, STANDARD_ATTN_S16 if s16 else 0, _ptr(workspace),
                           workspace.numel() * workspace.element_size(),
                           _stream(stream))
    _check(st, "standard_attn_bwd")
    return dq, dk, dv


# ---------------------------------------------------------------------------
# packed sequences with grouped heads, and serving from a paged cache
# ---------------------------------------------------------------------------
# These calls can take less time on the GPU than their checks take here, so the
# helpers look at each tensor once and build nothing twice.

FA_CACHE_16BIT, FA_CACHE_E4M3 = 0, 1
PACKED_DIRECT = 128          # a forward of so many sequences needs no workspace
# (int64 strides as bytes: packing them takes a tenth of a ctypes array's time)
_pack8, _pack16 = struct.Struct("=8q").pack, struct.Struct("=16q").pack
_pack_scores = struct.Struct("=IfQQ").pack     # fa_scores
_default_options = {}        # dtype -> (reference to) its fa_options
torch = None                 # bound with the library, by the first call


def _bind():
    """Loads the library and binds torch and the options, once."""
    global torch
    import torch as module
    lib = load()
    for dt, code in ((module.bfloat16, FA_DTYPE_BF16), (module.float16, FA_DTYPE_F16)):
        _default_options[dt] = ctypes.byref(fa_options(code))
    torch = module     # last: another thread's call that finds it finds the options too
    return lib


def _begin(t, wait_limit_us=0, test_stall=0):
    """The library, and (a reference to) the fa_options for t's dtype and the
    checking fields."""
    lib = _lib
    if lib is None or torch is None:
        lib = _bind()
    opts = _default_options.get(t.dtype)
    if opts is None or not t.is_cuda:
        raise ValueError("q (or k) must be a bfloat16 or float16 CUDA tensor")
    if wait_limit_us or test_stall:
        opts = ctypes.byref(fa_options(FA_DTYPE_F16 if t.dtype is torch.float16 else FA_DTYPE_BF16,
                                       wait_limit_us=wait_limit_us, test_stall=test_stall))
    return lib, opts


def _elsewhere(stream, dev):
    """None when a call launches on the current stream of the current device
    (dev), else the context to allocate and launch in."""
    if stream is None:
        if dev == torch._C._cuda_getDevice():
            return None
        return torch.cuda.stream(torch.cuda.current_stream(dev))
    if stream.device.index != dev:
        raise ValueError("the stream belongs to another device than the tensors")
    return torch.cuda.stream(stream)     # (also makes its device the current one)


def _rows16(t, name, shape, dtype, dev):
    """Checks a 16-bit tensor [tokens, heads, d] whose rows may be strided
    (views of a fused projection): d elements in one piece, token and head
    strides positive multiples of 8 elements. Returns the two strides."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev:
        raise ValueError(f"{name} must be a {dtype} tensor {list(shape)} on cuda:{dev}")
    tok, head, one = t.stride()
    if shape[0] <= 1:
        tok = shape[1] * shape[2]        # (the stride of a single token, or of none, says nothing)
    if shape[1] == 1:
        head = shape[2]
    if one != 1 or tok <= 0 or head <= 0 or (tok | head) & 7:
        raise ValueError(f"{name}: rows must be contiguous, with token and head strides that are positive multiples of 8")
    return tok, head


def _plain(t, name, shape, dtype, dev):
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {list(shape)} on cuda:{dev}")


def _past_32_bits():
    # (the C calls count in 32 bits, and ctypes would pass on what is left of a larger size)
    raise ValueError("a size does not fit 32 bits")


def _scratch(workspace, need, dev):
    """The caller's workspace, or a new one: (tensor, bytes)."""
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=dev), need
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"the workspace must be a contiguous tensor on cuda:{dev}")
    return workspace, workspace.numel() * workspace.element_size()


def _scores(softcap, slopes, prefix_lens, Hq, B, dev):
    """The fa_scores of a call as bytes."""
    cap = ctypes.c_float(softcap).value
    if softcap and not cap:              # (0 would be none at all)
        raise FlashAttnError(2 if softcap > 0 else 1, "softcap")
    if slopes is not None:
        _plain(slopes, "slopes", (Hq,), torch.float32, dev)
    if prefix_lens is not None:
        _plain(prefix_lens, "prefix_lens", (B,), torch.int32, dev)
    return _pack_scores(24, cap, 0 if slopes is None else slopes.data_ptr(),
                        0 if prefix_lens is None else prefix_lens.data_ptr())


def attention_packed_fwd(q, k, v, cu_seqlens, scale, causal=True, out=None, lse=None, workspace=None, stream=None,
                         wait_limit_us=0, test_stall=0, softcap=0.0, slopes=None, prefix_lens=None):
    """O, LSE of attention within each sequence of a packed batch. q: bf16 or
    fp16 [tokens, Hq, d]; k, v: [tokens, Hk, d], Hq a multiple of Hk (query
    head h reads key/value head h // (Hq // Hk)); rows may be strided, as views
    of a fused projection are. cu_seqlens: int32 [B + 1], sequence b is rows
    cu_seqlens[b] .. cu_seqlens[b + 1] - 1. Returns O like q and LSE float32
    [Hq, tokens]; rows of no sequence are left as they are in `out` and `lse`.
    softcap > 0 caps the scores: softcap * tanh(score / softcap). slopes, float32
    [Hq], lowers those of head h by slopes[h] times the distance of query and key.
    prefix_lens, int32 [B], lets all tokens of a sequence see its first
    prefix_lens[b] (causal calls only)."""
    lib, opts = _begin(q, wait_limit_us, test_stall)
    dev = q.get_device()
    ctx = _elsewhere(stream, dev)
    if ctx is not None:
        with ctx:
            return attention_packed_fwd(q, k, v, cu_seqlens, scale, causal, out, lse, workspace, None, wait_limit_us,
                                        test_stall, softcap, slopes, prefix_lens)
    dt = q.dtype
    if q.dim() != 3 or k.dim() != 3 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("q must be [tokens, Hq, d], k and v [tokens, Hk, d], cu_seqlens [B + 1]")
    T, Hq, d = q.shape
    Hk, B = k.shape[1], cu_seqlens.numel() - 1
    if (T | Hq | Hk | d | B) >> 31:
        _past_32_bits()
    _plain(cu_seqlens, "cu_seqlens", (B + 1,), torch.int32, dev)
    if out is None:
        out = torch.empty((T, Hq, d), dtype=dt, device=dev)
    if lse is None:
        lse = torch.empty((Hq, T), dtype=torch.float32, device=dev)
    else:
        _plain(lse, "lse", (Hq, T), torch.float32, dev)
    st = _pack8(*_rows16(q, "q", (T, Hq, d), dt, dev), *_rows16(k, "k", (T, Hk, d), dt, dev),
                *_rows16(v, "v", (T, Hk, d), dt, dev), *_rows16(out, "out", (T, Hq, d), dt, dev))
    ws, nbytes = None, 0
    if B > PACKED_DIRECT or workspace is not None:
        workspace, nbytes = _scratch(workspace, lib.flash_attn_packed_workspace_size(B, T, Hq, Hk, d, 0), dev)
        ws = workspace.data_ptr()
    if softcap or slopes is not None or prefix_lens is not None:
        rc = lib.flash_attn_packed_scored_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                                              cu_seqlens.data_ptr(), B, T, Hq, Hk, d, st, scale, 1 if causal else 0,
                                              _scores(softcap, slopes, prefix_lens, Hq, B, dev), opts, ws, nbytes,
                                              torch._C._cuda_getCurrentRawStream(dev))
        _check(rc, "flash_attn_packed_scored_fwd")
        return out, lse
    rc = lib.flash_attn_packed_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                                   cu_seqlens.data_ptr(), B, T, Hq, Hk, d, st, scale, 1 if causal else 0, opts, ws,
                                   nbytes, torch._C._cuda_getCurrentRawStream(dev))
    _check(rc, "flash_attn_packed_fwd")
    return out, lse


def attention_packed_bwd(q, k, v, o, do, lse, cu_seqlens, scale, causal=True, workspace=None, dq=None, dk=None, dv=None,
                         stream=None, wait_limit_us=0, test_stall=0, softcap=0.0, slopes=None, prefix_lens=None):
    """dQ, dK, dV of attention_packed_fwd from its inputs, its O and LSE and the
    output gradient do (like q); dK and dV are summed over the query heads that
    share a key/value head. Rows of no sequence are left as they are in dq, dk,
    dv (which may be strided like q, k, v). softcap, slopes (which get no gradient)
    and prefix_lens as in the forward call."""
    lib, opts = _begin(q, wait_limit_us, test_stall)
    dev = q.get_device()
    ctx = _elsewhere(stream, dev)
    if ctx is not None:
        with ctx:
            return attention_packed_bwd(q, k, v, o, do, lse, cu_seqlens, scale, causal, workspace, dq, dk, dv, None,
                                        wait_limit_us, test_stall, softcap, slopes, prefix_lens)
    dt = q.dtype
    if q.dim() != 3 or k.dim() != 3 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("q must be [tokens, Hq, d], k and v [tokens, Hk, d], cu_seqlens [B + 1]")
    T, Hq, d = q.shape
    Hk, B = k.shape[1], cu_seqlens.numel() - 1
    if (T | Hq | Hk | d | B) >> 31:
        _past_32_bits()
    hq, hk = (T, Hq, d), (T, Hk, d)
    _plain(cu_seqlens, "cu_seqlens", (B + 1,), torch.int32, dev)
    _plain(lse, "lse", (Hq, T), torch.float32, dev)
    if dq is None:
        dq = torch.empty(hq, dtype=dt, device=dev)
    if dk is None:
        dk = torch.empty(hk, dtype=dt, device=dev)
    if dv is None:
        dv = torch.empty(hk, dtype=dt, device=dev)
    st = _pack16(*_rows16(q, "q", hq, dt, dev), *_rows16(k, "k", hk, dt, dev), *_rows16(v, "v", hk, dt, dev),
                 *_rows16(o, "o", hq, dt, dev), *_rows16(do, "do", hq, dt, dev), *_rows16(dq, "dq", hq, dt, dev),
                 *_rows16(dk, "dk", hk, dt, dev), *_rows16(dv, "dv", hk, dt, dev))
    workspace, nbytes = _scratch(workspace, lib.flash_attn_packed_workspace_size(B, T, Hq, Hk, d, 1), dev)
    if softcap or slopes is not None or prefix_lens is not None:
        rc = lib.flash_attn_packed_scored_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(),
                                              lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                                              cu_seqlens.data_ptr(), B, T, Hq, Hk, d, st, scale, 1 if causal else 0,
                                              _scores(softcap, slopes, prefix_lens, Hq, B, dev), opts,
                                              workspace.data_ptr(), nbytes, torch._C._cuda_getCurrentRawStream(dev))
        _check(rc, "flash_attn_packed_scored_bwd")
        return dq, dk, dv
    rc = lib.flash_attn_packed_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(),
                                   lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                                   cu_seqlens.data_ptr(), B, T, Hq, Hk, d, st, scale, 1 if causal else 0, opts,
                                   workspace.data_ptr(), nbytes, torch._C._cuda_getCurrentRawStream(dev))
    _check(rc, "flash_attn_packed_bwd")
    return dq, dk, dv


def _cache_args(k_cache, v_cache, k_scale, v_scale, dtype, dev):
    """Checks the tensors of a paged cache; returns the cache type."""
    if k_cache.dim() != 4:
        raise ValueError("k_cache and v_cache must be [num_pages, Hk, page_size, d]")
    shape, kind = k_cache.shape, k_cache.dtype
    e4m3 = kind is torch.float8_e4m3fn
    if not e4m3 and kind is not dtype:
        raise ValueError("the cache must hold the 16-bit type of the other tensors, or float8_e4m3fn")
    _plain(k_cache, "k_cache", shape, kind, dev)
    _plain(v_cache, "v_cache", shape, kind, dev)
    if (k_scale is not None) != e4m3 or (v_scale is not None) != e4m3:
        raise ValueError("k_scale and v_scale belong to a float8_e4m3fn cache")
    if e4m3:
        _plain(k_scale, "k_scale", shape[:3], torch.float32, dev)
        _plain(v_scale, "v_scale", shape[:3], torch.float32, dev)
        return FA_CACHE_E4M3
    return FA_CACHE_16BIT


def kv_cache_write(k, v, slots, k_cache, v_cache, k_scale=None, v_scale=None, stream=None):
    """Writes keys and values k, v [T, Hk, d] (bf16 or fp16, rows may be
    strided) into a paged cache k_cache, v_cache [num_pages, Hk, page_size, d]:
    token t into place slots[t] % page_size of page slots[t] // page_size
    (int64; a slot outside the cache, -1 for instance, skips its token). A
    cache of the tokens' dtype takes them as they are; a float8_e4m3fn cache
    takes them quantised, with one power-of-two scale per row in k_scale,
    v_scale (float32 [num_pages, Hk, page_size])."""
    lib, opts = _begin(k)
    dev = k.get_device()
    ctx = _elsewhere(stream, dev)
    if ctx is not None:
        with ctx:
            return kv_cache_write(k, v, slots, k_cache, v_cache, k_scale, v_scale)
    dt = k.dtype
    kind = _cache_args(k_cache, v_cache, k_scale, v_scale, dt, dev)
    pages, Hk, page, d = k_cache.shape
    if k.dim() != 3:
        raise ValueError("k and v must be [T, Hk, d]")
    T = k.shape[0]
    if (T | pages | Hk | page | d) >> 31:
        _past_32_bits()
    k_tok, k_head = _rows16(k, "k", (T, Hk, d), dt, dev)
    v_tok, v_head = _rows16(v, "v", (T, Hk, d), dt, dev)
    _plain(slots, "slots", (T,), torch.int64, dev)
    e4m3 = kind == FA_CACHE_E4M3
    rc = lib.flash_attn_kv_cache_write(k.data_ptr(), v.data_ptr(), k_tok, k_head, v_tok, v_head, slots.data_ptr(), T,
                                       Hk, d, k_cache.data_ptr(), v_cache.data_ptr(),
                                       k_scale.data_ptr() if e4m3 else None, v_scale.data_ptr() if e4m3 else None,
                                       pages, page, kind, opts, torch._C._cuda_getCurrentRawStream(dev))
    _check(rc, "flash_attn_kv_cache_write")


def _newest(q, block_table, seq_lens, cache_shape, dev):
    """Checks the queries of the newest tokens and their sequences against a
    cache of this shape; returns B, Nq, Hq, the table's width, the token stride."""
    pages, Hk, page, d = cache_shape
    if q.dim() != 4 or q.shape[3] != d or block_table.dim() != 2:
        raise ValueError("q must be [B, Nq, Hq, d] with the cache's d, block_table [B, max_pages]")
    B, Nq, Hq, _ = q.shape
    width = block_table.shape[1]
    if (B | Nq | Hq | width | pages | Hk | page | d) >> 31:
        _past_32_bits()
    s0, s1, s2, s3 = q.stride()
    if s3 != 1 or (Hq > 1 and s2 != d) or (B > 1 and Nq > 1 and s0 != Nq * s1):
        raise ValueError("q: a token's heads must be contiguous and the tokens evenly spaced")
    _plain(block_table, "block_table", (B, width), torch.int32, dev)
    _plain(seq_lens, "seq_lens", (B,), torch.int32, dev)
    return B, Nq, Hq, width, s1 if Nq > 1 else (s0 if B > 1 else Hq * d)


def attention_cached_fwd(q, k_cache, v_cache, block_table, seq_lens, scale, k_scale=None, v_scale=None, out=None,
                         lse=None, workspace=None, stream=None, wait_limit_us=0, test_stall=0, softcap=0.0,
                         slopes=None):
    """O, LSE of the newest Nq tokens of B sequences against their keys and
    values in a paged cache. q: bf16 or fp16 [B, Nq, Hq, d] (a token's heads
    contiguous, tokens may be strided); the cache, its scales and the slots'
    meaning as in kv_cache_write; block_table int32 [B, max_pages]; seq_lens
    int32 [B] counts each sequence's tokens, the newest Nq included. Token i of
    the Nq sees seq_lens - (Nq - 1 - i) keys; query head h reads key/value head
    h // (Hq // Hk). Returns O like q (contiguous) and LSE float32 [B, Hq, Nq].
    softcap > 0 caps the scores: softcap * tanh(score / softcap). slopes, float32
    [Hq], lowers those of head h by slopes[h] times the distance of query and key."""
    lib, opts = _begin(q, wait_limit_us, test_stall)
    dev = q.get_device()
    ctx = _elsewhere(stream, dev)
    if ctx is not None:
        with ctx:
            return attention_cached_fwd(q, k_cache, v_cache, block_table, seq_lens, scale, k_scale, v_scale, out, lse,
                                        workspace, None, wait_limit_us, test_stall, softcap, slopes)
    dt = q.dtype
    kind = _cache_args(k_cache, v_cache, k_scale, v_scale, dt, dev)
    pages, Hk, page, d = k_cache.shape
    B, Nq, Hq, width, tok = _newest(q, block_table, seq_lens, k_cache.shape, dev)
    if out is None:
        out = torch.empty((B, Nq, Hq, d), dtype=dt, device=dev)
    else:
        _plain(out, "out", (B, Nq, Hq, d), dt, dev)
    if lse is None:
        lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=dev)
    else:
        _plain(lse, "lse", (B, Hq, Nq), torch.float32, dev)
    ws, nbytes = None, 0
    if workspace is not None or lib.flash_attn_cached_needs_workspace(B, Nq, Hq, Hk, d, page, width, kind):
        workspace, nbytes = _scratch(workspace, lib.flash_attn_cached_workspace_size(B, Nq, Hq, Hk, d), dev)
        ws = workspace.data_ptr()
    e4m3 = kind == FA_CACHE_E4M3
    if softcap or slopes is not None:
        rc = lib.flash_attn_cached_scored_fwd(q.data_ptr(), tok, k_cache.data_ptr(), v_cache.data_ptr(),
                                              k_scale.data_ptr() if e4m3 else None, v_scale.data_ptr() if e4m3 else None,
                                              block_table.data_ptr(), seq_lens.data_ptr(), out.data_ptr(),
                                              lse.data_ptr(), B, Nq, Hq, Hk, d, pages, page, width, scale, kind,
                                              _scores(softcap, slopes, None, Hq, B, dev), opts, ws, nbytes,
                                              torch._C._cuda_getCurrentRawStream(dev))
        _check(rc, "flash_attn_cached_scored_fwd")
        return out, lse
    rc = lib.flash_attn_cached_fwd(q.data_ptr(), tok, k_cache.data_ptr(), v_cache.data_ptr(),
                                   k_scale.data_ptr() if e4m3 else None, v_scale.data_ptr() if e4m3 else None,
                                   block_table.data_ptr(), seq_lens.data_ptr(), out.data_ptr(), lse.data_ptr(), B, Nq, Hq,
                                   Hk, d, pages, page, width, scale, kind, opts, ws, nbytes, torch._C._cuda_getCurrentRawStream(dev))
    _check(rc, "flash_attn_cached_fwd")
    return out, lse


def attention_cached_weights(q, k_cache, block_table, seq_lens, lse, scale, weights, k_scale=None, past=None,
                             stream=None, wait_limit_us=0, test_stall=0, softcap=0.0, slopes=None):
    """What each cached token received from the newest Nq tokens of its sequence,
    per key/value head, added to what it had before: into weights, float32
    [num_pages, Hk, page_size] like the scales of a cache, goes past (the same
    shape, weights itself perhaps; None: nothing) plus the sum over the queries
    and the heads of a group of exp(score - lse). The newest Nq tokens have no
    past. q, the keys' cache, block_table, seq_lens, scale, softcap and slopes as
    in attention_cached_fwd, lse float32 [B, Hq, Nq] from it. Places of no token
    are left as they are. Returns weights."""
    lib, opts = _begin(q, wait_limit_us, test_stall)
    dev = q.get_device()
    ctx = _elsewhere(stream, dev)
    if ctx is not None:
        with ctx:
            return attention_cached_weights(q, k_cache, block_table, seq_lens, lse, scale, weights, k_scale, past, None,
                                            wait_limit_us, test_stall, softcap, slopes)
    kind = _cache_args(k_cache, k_cache, k_scale, k_scale, q.dtype, dev)
    pages, Hk, page, d = k_cache.shape
    B, Nq, Hq, width, tok = _newest(q, block_table, seq_lens, k_cache.shape, dev)
    _plain(lse, "lse", (B, Hq, Nq), torch.float32, dev)
    _plain(weights, "weights", (pages, Hk, page), torch.float32, dev)
    if past is not None:
        _plain(past, "past", (pages, Hk, page), torch.float32, dev)
    rc = lib.flash_attn_cached_weights(q.data_ptr(), tok, k_cache.data_ptr(),
                                       k_scale.data_ptr() if kind == FA_CACHE_E4M3 else None, block_table.data_ptr(),
                                       seq_lens.data_ptr(), lse.data_ptr(), None if past is None else past.data_ptr(),
                                       weights.data_ptr(), B, Nq, Hq, Hk, d, pages, page, width, scale, kind,
                                       _scores(softcap, slopes, None, Hq, B, dev), opts,
                                       torch._C._cuda_getCurrentRawStream(dev))
    _check(rc, "flash_attn_cached_weights")
    return weights


def kv_cache_evict(k_cache, v_cache, weights, block_table, seq_lens, new_table, budget, recent, k_scale=None,
                   v_scale=None, new_lens=None, kept=None, stream=None):
    """Shortens B cached sequences to at most budget tokens for each key/value
    head: their `recent` newest and the others with the largest weights (float32
    [num_pages, Hk, page_size], see attention_cached_weights; of equal ones the
    earlier). Those that stay keep their order and are copied, with their scales
    and weights, to the pages of new_table (int32 [B, new_pages]), which must be in
    no block_table; the old pages are only read. Returns the new lengths, int32
    [B], and the kept tokens' former places, int32 [B, Hk, budget], -1 past them."""
    lib = _lib
    if lib is None or torch is None:
        lib = _bind()
    if not weights.is_cuda or (k_cache.dtype not in _default_options and k_cache.dtype is not torch.float8_e4m3fn):
        raise ValueError("the cache must be bfloat16, float16 or float8_e4m3fn, and weights a CUDA tensor")
    dev = weights.get_device()
    ctx = _elsewhere(stream, dev)
    if ctx is not None:
        with ctx:
            return kv_cache_evict(k_cache, v_cache, weights, block_table, seq_lens, new_table, budget, recent, k_scale,
                                  v_scale, new_lens, kept)
    kind = _cache_args(k_cache, v_cache, k_scale, v_scale, k_cache.dtype, dev)
    pages, Hk, page, d = k_cache.shape
    if block_table.dim() != 2 or new_table.dim() != 2:
        raise ValueError("block_table must be [B, max_pages], new_table [B, new_pages]")
    B, width = block_table.shape
    new_width = new_table.shape[1]
    budget, recent = int(budget), int(recent)
    if (B | width | new_width | pages | Hk | page | d | max(budget, 0) | max(recent, 0)) >> 31:
        _past_32_bits()
    if budget < 1 or not 0 <= recent <= budget:
        raise ValueError("budget must be at least 1 and recent between 0 and it")
    _plain(weights, "weights", (pages, Hk, page), torch.float32, dev)
    _plain(block_table, "block_table", (B, width), torch.int32, dev)
    _plain(new_table, "new_table", (B, new_width), torch.int32, dev)
    _plain(seq_lens, "seq_lens", (B,), torch.int32, dev)
    if new_lens is None:
        new_lens = torch.empty(B, dtype=torch.int32, device=dev)
    else:
        _plain(new_lens, "new_lens", (B,), torch.int32, dev)
    if kept is None:
        kept = torch.empty((B, Hk, budget), dtype=torch.int32, device=dev)
    else:
        _plain(kept, "kept", (B, Hk, budget), torch.int32, dev)
    e4m3 = kind == FA_CACHE_E4M3
    rc = lib.flash_attn_kv_cache_evict(k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr() if e4m3 else None,
                                       v_scale.data_ptr() if e4m3 else None, weights.data_ptr(), block_table.data_ptr(),
                                       seq_lens.data_ptr(), new_table.data_ptr(), new_lens.data_ptr(), kept.data_ptr(),
                                       B, Hk, d, pages, page, width, new_width, budget, recent, kind, None,
                                       torch._C._cuda_getCurrentRawStream(dev))
    _check(rc, "flash_attn_kv_cache_evict")
    return new_lens, kept
