"""Refusals of the paged-cache calls, decided on the host before any launch:
the C ABI's argument checks (with pointers that are never dereferenced) and
the tensor checks of the Python helpers that need no GPU."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def L():
    from exact_io_aware_39_gb300 import build as b
    import exact_io_aware_39_gb300._lib as lib
    lib.load(b.build())
    return lib


P = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 8)


def _write(L, K=P, V=P, kt=1024, kh=128, vt=1024, vh=128, slots=P, T=4, Hk=8, d=128, kc=P, vc=P, ks=None, vs=None,
           pages=10, page=16, kind=0, opts=None):
    return L.flash_attn_kv_cache_write(K, V, kt, kh, vt, vh, slots, T, Hk, d, kc, vc, ks, vs, pages, page, kind, opts, None)


@pytest.mark.parametrize("kw,want", [
    (dict(K=None), 1), (dict(V=ODD), 1), (dict(slots=None), 1), (dict(slots=ctypes.c_void_p((1 << 20) + 4)), 1),
    (dict(kc=None), 1), (dict(vc=ODD), 1), (dict(T=-1), 1), (dict(Hk=0), 1), (dict(pages=0), 1),
    (dict(kt=1028), 1), (dict(vh=4), 1), (dict(d=0), 2), (dict(d=60), 2), (dict(d=136), 2), (dict(page=8), 2),
    (dict(page=48), 2), (dict(page=512), 2), (dict(kind=2), 2), (dict(ks=P, vs=P), 1),
    (dict(kind=1), 1), (dict(kind=1, ks=P), 1), (dict(kind=1, ks=P, vs=ODD), 1), (dict(kind=1, ks=P, vs=P, d=72), 2),
    (dict(T=1 << 24, Hk=8), 2), (dict(Hk=1025), 2),
])
def test_write_refusals(L, kw, want):
    assert _write(L, **kw) == want


def test_write_of_no_tokens_is_no_launch(L):
    assert _write(L, T=0, K=None, V=None, slots=None) == 0


def test_write_options(L):
    assert _write(L, opts=L.fa_options(7)) == 2
    assert _write(L, opts=L.fa_options(p_drop=0.1)) == 2
    assert _write(L, opts=L.fa_options(tile_record=1 << 20)) == 2


def _cached(L, Q=P, tok=4096, kc=P, vc=P, ks=None, vs=None, table=P, lens=P, O=P, LSE=P, B=2, Nq=1, Hq=32, Hk=8, d=128,
            pages=10, page=16, max_pages=4, scale=0.1, kind=0, opts=None, ws=P, nbytes=None):
    if nbytes is None:
        nbytes = L.flash_attn_cached_workspace_size(2, 1, 32, 8, 128)
    return L.flash_attn_cached_fwd(Q, tok, kc, vc, ks, vs, table, lens, O, LSE, B, Nq, Hq, Hk, d, pages, page, max_pages,
                                   scale, kind, opts, ws, nbytes, None)


@pytest.mark.parametrize("kw,want", [
    (dict(Q=None), 1), (dict(Q=ODD), 1), (dict(kc=ODD), 1), (dict(table=None), 1), (dict(lens=None), 1),
    (dict(O=ODD), 1), (dict(LSE=None), 1), (dict(B=0), 1), (dict(Nq=0), 1), (dict(Hq=31), 1), (dict(Hk=0), 1),
    (dict(max_pages=0), 1), (dict(pages=0), 1), (dict(scale=0.0), 1), (dict(scale=-0.5), 1),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(tok=4100), 1), (dict(tok=4088), 1),
    (dict(d=132), 2), (dict(d=136, tok=8192), 2), (dict(page=12), 2), (dict(kind=3), 2), (dict(kind=1), 1),
    (dict(ks=P), 1), (dict(kind=1, ks=P, vs=P, d=120), 2), (dict(pages=1 << 30), 2), (dict(max_pages=1 << 27), 2),
    (dict(B=1 << 20, Nq=64), 2),
])
def test_cached_refusals(L, kw, want):
    assert _cached(L, **kw) == want


def test_cached_workspace(L):
    need = L.flash_attn_cached_workspace_size(2, 1, 32, 8, 128)
    def al(x):
        return (x + 255) // 256 * 256
    assert need == al(al(1824 * 2 * 16 * 128 * 4) + 1824 * 2 * 16 * 8) + al(2 * 8 * 8)
    assert _cached(L, nbytes=need - 1) == 3
    # a table of 4 pages of 16: joined on chip, no workspace needed; of 4096 pages: needed
    assert L.flash_attn_cached_needs_workspace(2, 1, 32, 8, 128, 16, 4, 0) == 0
    assert L.flash_attn_cached_needs_workspace(2, 1, 32, 8, 128, 16, 4096, 0) == 1
    assert L.flash_attn_cached_needs_workspace(64, 1, 32, 8, 128, 16, 4, 0) == 1
    assert _cached(L, ws=None, max_pages=4096) == 3
    assert _cached(L, ws=ctypes.c_void_p((1 << 20) + 16)) == 3
    for bad in ((0, 1, 32, 8, 128), (1, 0, 32, 8, 128), (1, 1, 30, 8, 128), (1, 1, 8, 8, 130), (1, 1, 8, 8, 256)):
        assert L.flash_attn_cached_workspace_size(*bad) == 0


def test_cached_options(L):
    assert _cached(L, opts=L.fa_options(p_drop=0.1)) == 2
    assert _cached(L, opts=L.fa_options(tile_record=1 << 20)) == 2
    assert _cached(L, opts=L.fa_options(test_stall=2)) == 1


def test_helpers_refuse_cpu_tensors(L):
    k = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    c = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        L.kv_cache_write(k, k, torch.arange(4), c, c)
    with pytest.raises(ValueError):
        L.attention_cached_fwd(k[:, None], c, c, torch.zeros(4, 1, dtype=torch.int32),
                               torch.ones(4, dtype=torch.int32), 0.1)


def test_write_refuses_a_stall(L):
    """(it has no wait that could run out)"""
    assert _write(L, opts=L.fa_options(test_stall=1)) == 2
    assert _write(L, opts=L.fa_options(test_stall=2)) == 1
