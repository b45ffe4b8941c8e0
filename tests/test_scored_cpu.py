"""Refusals of the calls with capped or biased scores, decided on the host
before any launch."""
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


def _calls(L, scores, scale=0.1, causal=1, P=P, **kw):
    a = dict(B=2, total=300, Hq=8, Hk=2, d=128, st=None, opts=None, ws=P, nbytes=1 << 40)
    a.update(kw)
    yield L.flash_attn_packed_scored_fwd(P, P, P, P, P, P, a["B"], a["total"], a["Hq"], a["Hk"], a["d"], a["st"], scale,
                                         causal, scores, a["opts"], a["ws"], a["nbytes"], None)
    yield L.flash_attn_packed_scored_bwd(P, P, P, P, P, P, P, P, P, P, a["B"], a["total"], a["Hq"], a["Hk"], a["d"],
                                         a["st"], scale, causal, scores, a["opts"], a["ws"], a["nbytes"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(softcap=-1.0), 1), (dict(softcap=float("nan")), 1), (dict(softcap=float("inf")), 1),
    (dict(softcap=2.0 ** -11), 2), (dict(softcap=1025.0), 2), (dict(slopes=(1 << 20) + 2), 1),
    (dict(prefix_lens=(1 << 20) + 1), 1),
])
def test_scores_that_are_refused(L, kw, want):
    for st in _calls(L, L.fa_scores(**kw)):
        assert st == want


def test_scores_and_other_arguments(L):
    pre = L.fa_scores(prefix_lens=1 << 20)
    for st in _calls(L, pre, causal=0):
        assert st == 1
    for st in _calls(L, L.fa_scores(softcap=30.0), scale=2.0 ** 80):
        assert st == 2                                    # scale / softcap leaves the fp32 range, squared
    short = L.fa_scores(softcap=-1.0)
    short.size = 8                                        # a caller of an older struct: softcap is read
    for st in _calls(L, short):
        assert st == 1
    short.size = 4
    short.softcap = 30.0
    for st in _calls(L, short):
        assert st == 1
    # what the plain calls refuse
    ok = L.fa_scores(softcap=30.0)
    for kw, want in ((dict(B=-1), 1), (dict(Hq=9), 1), (dict(d=12), 2), (dict(ws=ctypes.c_void_p(16)), 3),
                     (dict(opts=L.fa_options(p_drop=0.1)), 2), (dict(scale=0.0), 1), (dict(causal=2), 1)):
        for st in _calls(L, ok, **kw):
            assert st == want, kw
    for st in _calls(L, ok, B=0, P=None, ws=None, nbytes=0):
        assert st == 0


def test_helpers_refuse_cpu_tensors(L):
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError):
        L.attention_packed_fwd(q, q, q, cu, 0.1, softcap=30.0)


ODD = ctypes.c_void_p((1 << 20) + 4)


def _cached(L, scores=None, Q=P, kc=P, vc=P, table=P, lens=P, LSE=P, **kw):
    a = dict(tok=4096, B=2, Nq=1, Hq=32, Hk=8, d=128, pages=10, page=16, width=4, scale=0.1, kind=0, ks=None, opts=None)
    a.update(kw)
    vs = a["ks"]
    yield L.flash_attn_cached_scored_fwd(Q, a["tok"], kc, vc, a["ks"], vs, table, lens, P, LSE, a["B"], a["Nq"], a["Hq"],
                                         a["Hk"], a["d"], a["pages"], a["page"], a["width"], a["scale"], a["kind"],
                                         scores, a["opts"], P, 1 << 40, None)
    yield L.flash_attn_cached_weights(Q, a["tok"], kc, a["ks"], table, lens, LSE, None, vc, a["B"], a["Nq"], a["Hq"],
                                      a["Hk"], a["d"], a["pages"], a["page"], a["width"], a["scale"], a["kind"], scores,
                                      a["opts"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(Q=None), 1), (dict(kc=ctypes.c_void_p((1 << 20) + 8)), 1), (dict(vc=ODD), 1), (dict(vc=None), 1),
    (dict(table=None), 1), (dict(lens=ctypes.c_void_p((1 << 20) + 2)), 1), (dict(LSE=None), 1), (dict(B=0), 1),
    (dict(Nq=0), 1), (dict(Hq=31), 1), (dict(scale=0.0), 1), (dict(kind=2), 2), (dict(kind=1), 1), (dict(ks=P), 1),
    (dict(kind=1, ks=P, d=72), 2), (dict(d=12), 2), (dict(page=24), 2), (dict(width=0), 1), (dict(tok=4095), 1),
    (dict(tok=2048), 1), (dict(pages=1 << 30), 2), (dict(width=1 << 27), 2),
])
def test_cached_refusals(L, kw, want):
    for st in _cached(L, **kw):
        assert st == want


def test_cached_scores_and_options(L):
    for kw, want in ((dict(softcap=-1.0), 1), (dict(softcap=1e9), 2), (dict(slopes=(1 << 20) + 1), 1),
                     (dict(prefix_lens=1 << 20), 2)):
        for st in _cached(L, scores=L.fa_scores(**kw)):
            assert st == want
    for opts, want in ((L.fa_options(7), 2), (L.fa_options(p_drop=0.1), 2), (L.fa_options(tile_record=1 << 20), 2),
                       (L.fa_options(test_stall=2), 1)):
        for st in _cached(L, opts=opts):
            assert st == want
    assert L.flash_attn_cached_weights(P, 4096, P, None, P, P, P, ODD, P, 2, 1, 32, 8, 128, 10, 16, 4, 0.1, 0, None, None,
                                       None) == 1       # past


def _evict(L, kc=P, vc=P, ks=None, vs=None, w=P, table=P, lens=P, new=P, nl=P, kept=P, B=2, Hk=8, d=128, pages=10, page=16,
           width=4, new_width=2, budget=32, recent=8, kind=0, opts=None):
    return L.flash_attn_kv_cache_evict(kc, vc, ks, vs, w, table, lens, new, nl, kept, B, Hk, d, pages, page, width,
                                       new_width, budget, recent, kind, opts, None)


@pytest.mark.parametrize("kw,want", [
    (dict(kc=None), 1), (dict(vc=ctypes.c_void_p((1 << 20) + 8)), 1), (dict(w=None), 1), (dict(table=None), 1),
    (dict(lens=None), 1), (dict(new=None), 1), (dict(nl=None), 1), (dict(kept=None), 1),
    (dict(kept=ctypes.c_void_p((1 << 20) + 2)), 1), (dict(B=0), 1), (dict(Hk=0), 1), (dict(pages=0), 1),
    (dict(width=0), 1), (dict(new_width=0), 1), (dict(budget=0), 1), (dict(budget=33), 1), (dict(recent=-1), 1),
    (dict(recent=33), 1), (dict(kind=2), 2), (dict(d=12), 2), (dict(d=136), 2), (dict(page=24), 2), (dict(ks=P, vs=P), 1),
    (dict(kind=1), 1), (dict(kind=1, ks=P), 1), (dict(kind=1, ks=P, vs=P, d=72), 2), (dict(width=1 << 27), 2),
    (dict(new_width=1 << 27, budget=1 << 20), 2), (dict(B=1 << 20, Hk=1 << 12), 2),
])
def test_evict_refusals(L, kw, want):
    assert _evict(L, **kw) == want


def test_evict_options(L):
    for opts, want in ((L.fa_options(7), 2), (L.fa_options(p_drop=0.1), 2), (L.fa_options(test_stall=1), 2)):
        assert _evict(L, opts=opts) == want


@pytest.mark.parametrize("softcap,status", [(1e-46, 2), (5e-324, 2), (-1e-46, 1)])
def test_helpers_refuse_a_cap_that_32_bits_make_none(L, softcap, status):
    with pytest.raises(L.FlashAttnError) as e:
        L._scores(softcap, None, None, 8, 2, 0)
    assert e.value.status == status


@pytest.mark.parametrize("softcap", [0.0, 2.0 ** -10, 30.0, 0.1, 1024.0, 5000.0, 1e39, float("inf"), -1e39])
def test_helpers_pack_the_scores_as_the_struct_does(L, softcap):
    """Also a cap that 32 bits make infinite, which the call refuses."""
    assert L._scores(softcap, None, None, 8, 2, 0) == bytes(L.fa_scores(softcap))
    if not 2.0 ** -10 <= softcap <= 1024.0 and softcap:
        for st in _calls(L, L.fa_scores(softcap)):
            assert st in (1, 2)
