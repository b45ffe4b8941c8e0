"""Refusals of the packed calls, decided on the host before any launch."""
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


def _strides(n, bad=None, value=None):
    s = [1024, 128] * n
    if bad is not None:
        s[bad] = value
    return (ctypes.c_int64 * (2 * n))(*s)


def _fwd(L, Q=P, K=P, V=P, O=P, LSE=P, cu=P, B=2, total=300, Hq=8, Hk=2, d=128, st=None, scale=0.1, causal=1, opts=None,
         ws=P, nbytes=None):
    if nbytes is None:
        nbytes = L.flash_attn_packed_workspace_size(2, 300, 8, 2, 128, 0)
    return L.flash_attn_packed_fwd(Q, K, V, O, LSE, cu, B, total, Hq, Hk, d, st, scale, causal, opts, ws, nbytes, None)


def _bwd(L, ptrs=None, LSE=P, cu=P, B=2, total=300, Hq=8, Hk=2, d=128, st=None, scale=0.1, causal=1, opts=None, ws=P,
         nbytes=None):
    q, k, v, o, do, dq, dk, dv = ptrs or [P] * 8
    if nbytes is None:
        nbytes = L.flash_attn_packed_workspace_size(2, 300, 8, 2, 128, 1)
    return L.flash_attn_packed_bwd(q, k, v, o, do, LSE, dq, dk, dv, cu, B, total, Hq, Hk, d, st, scale, causal, opts, ws,
                                   nbytes, None)


SHAPES = [
    (dict(B=-1), 1), (dict(total=-1), 1), (dict(Hk=0), 1), (dict(Hq=0), 1), (dict(Hq=9), 1), (dict(d=0), 2),
    (dict(d=12), 2), (dict(d=136), 2), (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(causal=2), 1), (dict(total=1 << 30, Hq=64), 2), (dict(B=1 << 30), 2),
    (dict(LSE=None), 1), (dict(cu=None), 1), (dict(cu=ctypes.c_void_p((1 << 20) + 2)), 1),
    (dict(ws=None, B=140), 3), (dict(ws=ctypes.c_void_p((1 << 20) + 16)), 3), (dict(nbytes=100), 3),
]


@pytest.mark.parametrize("kw,want", SHAPES)
def test_refusals(L, kw, want):
    assert _fwd(L, **kw) == want
    assert _bwd(L, **kw) == want


def test_pointers_and_strides(L):
    for name in "QKVO":
        assert _fwd(L, **{name: None}) == 1 and _fwd(L, **{name: ODD}) == 1
    for i in range(8):
        for x in (None, ODD):
            ptrs = [P] * 8
            ptrs[i] = x
            assert _bwd(L, ptrs) == 1
    for i in range(8):
        for v in (0, -128, 12, 1 << 36):
            assert _fwd(L, st=_strides(4, i, v)) == 1
    for i in range(16):
        for v in (0, -128, 12, 1 << 36):
            assert _bwd(L, st=_strides(8, i, v)) == 1


def test_nothing_to_do(L):
    for kw in (dict(B=0), dict(total=0)):
        assert _fwd(L, Q=None, K=None, V=None, O=None, LSE=None, cu=None, ws=None, nbytes=0, **kw) == 0
        assert _bwd(L, [None] * 8, LSE=None, cu=None, ws=None, nbytes=0, **kw) == 0


def test_options(L):
    for call in (_fwd, _bwd):
        assert call(L, opts=L.fa_options(7)) == 2
        assert call(L, opts=L.fa_options(p_drop=0.1)) == 2
        assert call(L, opts=L.fa_options(tile_record=1 << 20)) == 2
        assert call(L, opts=L.fa_options(test_stall=2)) == 1


def test_workspace_size(L):
    def al(x):
        return (x + 255) // 256 * 256
    B, total, Hq, d = 5, 1000, 8, 96
    tiles = total // 128 + B
    want = al(al(al(256) + 4 * B) + 16 * tiles)
    assert L.flash_attn_packed_workspace_size(B, total, Hq, 2, d, 0) == want
    # an odd group: two query tiles to an item
    assert L.flash_attn_packed_workspace_size(B, total, Hq, Hq, d, 0) == al(al(al(256) + 4 * B) + 16 * (total // 256 + B))
    want = al(al(al(256) + 4 * B) + 16 * tiles)
    want = al(want + 16 * tiles)
    rows = Hq * tiles * 128
    want = al(want + rows * d * 4)
    want = al(al(want + rows * 4) + rows * 4)
    # 24 items of 3 + 5 steps for 152 SMs: in as many parts as an item has steps
    # (4 heads, 2 tiles of an average sequence), each with its dK and dV
    part = 8 * 2 * 2 * tiles * 128 * d * 4
    assert L.flash_attn_packed_workspace_size(B, total, Hq, 2, d, 1) == al(want + part)
    # two items for every SM: no parts
    B, total, tiles, Hk = 5, 20000, 20000 // 128 + 5, 2
    rows = Hq * tiles * 128
    want = al(al(al(al(al(256) + 4 * B) + 16 * tiles) + 16 * tiles) + rows * d * 4)
    assert L.flash_attn_packed_workspace_size(B, total, Hq, Hk, d, 1) == al(al(want + rows * 4) + rows * 4)
    for bad in ((-1, 1, 1, 1, 64), (1, 1, 3, 2, 64), (1, 1, 1, 1, 256), (1, 1, 1, 1, 4)):
        assert L.flash_attn_packed_workspace_size(*bad, 0) == 0


def test_helpers_refuse_cpu_tensors(L):
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError):
        L.attention_packed_fwd(q, q, q, cu, 0.1)
    with pytest.raises(ValueError):
        L.attention_packed_bwd(q, q, q, q, q, torch.zeros(2, 4), cu, 0.1)


def test_first_calls_of_two_threads(L, monkeypatch):
    """A thread whose first call comes while another's prepares the helpers gets
    its options too."""
    import threading
    from types import SimpleNamespace
    monkeypatch.setattr(L, "torch", None)
    monkeypatch.setattr(L, "_default_options", {})
    make, got = L.fa_options, []
    tensors = [SimpleNamespace(dtype=dt, is_cuda=True) for dt in (torch.bfloat16, torch.float16)]

    def second():
        for t in tensors:
            try:
                got.append(L._begin(t))
            except ValueError as e:
                got.append(e)

    class Slowly(make):
        def __init__(self, *a, **kw):
            if threading.current_thread() is threading.main_thread():
                other = threading.Thread(target=second)
                other.start()
                other.join()
            super().__init__(*a, **kw)

    monkeypatch.setattr(L, "fa_options", Slowly)
    got.append(L._begin(tensors[0]))
    assert len(got) >= 3 and all(isinstance(x, tuple) and x[1] is not None for x in got), got


def test_sizes_past_32_bits_are_refused(L, monkeypatch):
    """The C calls count in 32 bits; a size of 2^32 and a bit must not arrive as
    the bit."""
    class Library:
        def __getattr__(self, name):
            raise AssertionError(f"{name} was called")

    monkeypatch.setattr(L, "torch", torch)
    monkeypatch.setattr(L, "_begin", lambda *a: (Library(), None))
    monkeypatch.setattr(L, "_elsewhere", lambda *a: None)
    far = (1 << 32) + 8
    mk = lambda *s, dtype=torch.bfloat16: torch.empty(*s, dtype=dtype, device="meta")
    i32, f32 = torch.int32, torch.float32
    for T, H, d in ((far, 1, 8), (8, far, 8), (8, 1, far)):
        x, lse = mk(T, H, d), mk(H, T, dtype=f32)
        cu = mk(3, dtype=i32)
        with pytest.raises(ValueError, match="32 bits"):
            L.attention_packed_fwd(x, x, x, cu, 0.1, out=x, lse=lse)
        with pytest.raises(ValueError, match="32 bits"):
            L.attention_packed_bwd(x, x, x, x, x, lse, cu, 0.1, dq=x, dk=x, dv=x)
    x, lse = mk(8, 1, 8), mk(1, 8, dtype=f32)
    with pytest.raises(ValueError, match="32 bits"):
        L.attention_packed_fwd(x, x, x, mk(far, dtype=i32), 0.1, out=x, lse=lse)
    for pages, T, d in ((4, far, 8), (far, 8, 8), (4, 8, far)):
        c, x = mk(pages, 1, 16, d), mk(T, 1, d)
        with pytest.raises(ValueError, match="32 bits"):
            L.kv_cache_write(x, x, mk(T, dtype=torch.int64), c, c)
    for B, Nq, Hq, width in ((far, 1, 1, 4), (2, far, 1, 4), (2, 1, far, 4), (2, 1, 1, far)):
        c, q = mk(4, 1, 16, 8), mk(B, Nq, Hq, 8)
        with pytest.raises(ValueError, match="32 bits"):
            L.attention_cached_fwd(q, c, c, mk(B, width, dtype=i32), mk(B, dtype=i32), 0.1, out=q,
                                   lse=mk(B, Hq, Nq, dtype=f32))
