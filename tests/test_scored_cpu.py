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
