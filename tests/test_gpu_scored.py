"""Attention with capped and biased scores and prefix masks on the GPU against
the float64 reference, element by element within the bounds that
oracle/scored.py derives from the roundings. Rows of no sequence hold NaN in
every input and a canary in every output."""
import numpy as np
import pytest
import torch

from oracle import scored as S
from test_gpu_packed import BF, CANARY, FH, _bits, _f64, _inputs, _outputs, _settled, fa  # noqa: F401 (fa: the fixture)
from test_gpu_packed import _check as packed_check

pytestmark = pytest.mark.gpu


def _score_args(lens, Hq, softcap, bias, prefix, seed=0):
    r = np.random.default_rng(seed)
    kw = dict(softcap=softcap)
    if bias:
        kw["slopes"] = torch.tensor(2.0 ** -r.uniform(0, 8, Hq), dtype=torch.float32, device="cuda")
    if prefix:
        pre = [int(r.integers(0, n + 1)) if i % 3 else (n, 0, -5, n + 9)[i // 3 % 4] for i, n in enumerate(lens)]
        kw["prefix_lens"] = torch.tensor(pre, dtype=torch.int32, device="cuda")
    return kw


def _run(fa, c, scale, causal, kw, out=None, ws=(None, None), **more):  # noqa: F811
    r = _outputs(c) if out is None else out
    fa.attention_packed_fwd(c["q"], c["k"], c["v"], c["cu"], scale, causal=causal, out=r["o"], lse=r["lse"],
                            workspace=ws[0], **kw, **more)
    fa.attention_packed_bwd(c["q"], c["k"], c["v"], r["o"], c["do"], r["lse"], c["cu"], scale, causal=causal,
                            dq=r["dq"], dk=r["dk"], dv=r["dv"], workspace=ws[1], **kw, **more)
    return r


def _check(c, r, scale, causal, kw, bounds=None):
    u = 2.0 ** -8 if c["q"].dtype == BF else 2.0 ** -11
    host = lambda x: None if x is None else x.cpu().numpy()
    val, tol = S.packed_attention(_f64(c["q"]), _f64(c["k"]), _f64(c["v"]), _f64(c["do"]),
                                  c["bounds"] if bounds is None else bounds, scale, causal, u, kw.get("softcap", 0.0),
                                  host(kw.get("slopes")), host(kw.get("prefix_lens")))
    for name, key in (("O", "o"), ("LSE", "lse"), ("dQ", "dq"), ("dK", "dk"), ("dV", "dv")):
        got, ref = _f64(r[key]), val[name]
        none = np.isnan(ref)
        assert (got[none] == CANARY).all(), f"{name}: rows of no sequence were written"
        assert np.isfinite(got).all(), f"{name} is not finite"
        over = np.abs(got[~none] - ref[~none]) - tol[name][~none]
        assert over.size == 0 or over.max() <= 0, f"{name}: {over.max():.3g} over its bound"


def _again(fa, c, r, scale, causal, kw):  # noqa: F811
    r2 = _run(fa, c, scale, causal, kw)
    _settled(fa)
    for key in ("o", "lse", "dk", "dv"):     # (dQ's partial sums are added as they come)
        assert torch.equal(_bits(r[key].contiguous()), _bits(r2[key].contiguous())), key


SHAPES = [
    # lens, Hq, Hk, d, before, behind, fused
    ([1], 1, 1, 64, 0, 0, False), ([128], 2, 2, 128, 0, 0, False), ([129, 2], 4, 1, 64, 0, 5, True),
    ([127, 1, 128, 256, 0, 3], 4, 2, 128, 3, 200, True), ([300, 0, 511], 6, 2, 64, 0, 1, False),
    ([640], 3, 1, 128, 1, 0, True), ([17, 40, 5, 60, 33], 8, 2, 80, 0, 130, False), ([250, 390], 4, 4, 40, 0, 0, True),
    ([200, 257], 2, 1, 8, 7, 9, False), ([70] * 30, 4, 2, 128, 0, 0, True),
]
KINDS = [
    # softcap, slopes, causal, prefix, q's factor (scores' size)
    (30.0, False, True, False, 1.0), (30.0, False, False, False, 20.0), (5.0, True, True, True, 4.0),
    (0.0, True, True, False, 1.0), (0.0, True, False, False, 1.0), (0.0, True, True, True, 1.0),
    (0.0, False, True, True, 1.0), (50.0, True, False, False, 10.0), (50.0, False, True, True, 3.0),
]


@pytest.mark.parametrize("dtype", [BF, FH], ids=["bf16", "fp16"])
@pytest.mark.parametrize("softcap,bias,causal,prefix,qmul", KINDS)
@pytest.mark.parametrize("lens,Hq,Hk,d,before,behind,fused", SHAPES)
def test_forward_and_gradients(fa, lens, Hq, Hk, d, before, behind, fused, softcap, bias, causal, prefix, qmul, dtype):  # noqa: F811
    c = _inputs(lens, Hq, Hk, d, dtype, len(lens), before, behind, fused, qmul)
    kw = _score_args(lens, Hq, softcap, bias, prefix, d)
    scale = d ** -0.5
    r = _run(fa, c, scale, causal, kw)
    _settled(fa)
    _check(c, r, scale, causal, kw)


@pytest.mark.parametrize("softcap,qmul", [(2.0 ** -10, 1.0), (0.5, 1.0), (1024.0, 1.0), (1024.0, 200.0), (20.0, 5.0)])
@pytest.mark.parametrize("d", [64, 128])
def test_caps_of_all_sizes(fa, d, softcap, qmul):  # noqa: F811
    c = _inputs([200, 77], 2, 1, d, FH, 3, 0, 3, qmul=qmul)
    r = _run(fa, c, d ** -0.5, True, dict(softcap=softcap))
    _settled(fa)
    _check(c, r, d ** -0.5, True, dict(softcap=softcap))


def test_scores_past_the_exponential(fa):  # noqa: F811
    """Scores of thousands: the cap's exponential overflows and vanishes."""
    c = _inputs([150], 2, 2, 64, FH, 4, qmul=100.0)
    c["k"] = (c["k"].float() * 100).half()
    r = _run(fa, c, 1.0, True, dict(softcap=15.0))
    _settled(fa)
    _check(c, r, 1.0, True, dict(softcap=15.0))


@pytest.mark.parametrize("B", [33, 128, 129, 140])
@pytest.mark.parametrize("Hq,Hk,d,kind", [(2, 2, 64, 5), (4, 2, 128, 2), (3, 1, 128, 6)])
def test_many_sequences(fa, Hq, Hk, d, kind, B):  # noqa: F811
    """Lists of several sequences to a lane, and those of the plan kernel, with
    prefixes in them."""
    lens = [(97 * b) % 301 for b in range(B)]
    softcap, bias, causal, prefix, qmul = KINDS[kind]
    c = _inputs(lens, Hq, Hk, d, BF, 8, 2, 70, qmul=qmul)
    kw = _score_args(lens, Hq, softcap, bias, prefix, 1)
    r = _run(fa, c, d ** -0.5, causal, kw)
    _settled(fa)
    _check(c, r, d ** -0.5, causal, kw)


@pytest.mark.parametrize("kind", [0, 2, 5, 6])
@pytest.mark.parametrize("lens,Hq,Hk,d", [([300, 140, 1000, 128, 1], 12, 3, 128), ([1300], 14, 7, 64),
                                          ([400, 300, 129, 77, 128, 1, 0, 250, 513], 32, 16, 64),
                                          ([900], 1, 1, 64), ([260], 7, 1, 64), ([2300, 700], 2, 1, 128)])
def test_items_alone_whole_and_in_parts(fa, lens, Hq, Hk, d, kind):  # noqa: F811
    """Query tiles on their own, items of the backward that stay whole (16 heads)
    and in parts; results repeat bit for bit."""
    softcap, bias, causal, prefix, qmul = KINDS[kind]
    c = _inputs(lens, Hq, Hk, d, BF, 15, 2, 9, True, qmul)
    kw = _score_args(lens, Hq, softcap, bias, prefix, 2)
    r = _run(fa, c, d ** -0.5, causal, kw)
    _settled(fa)
    _check(c, r, d ** -0.5, causal, kw)
    _again(fa, c, r, d ** -0.5, causal, kw)


def test_slopes_of_any_sign(fa):  # noqa: F811
    lens = [200, 131]
    c = _inputs(lens, 4, 2, 64, BF, 10)
    kw = dict(slopes=torch.tensor([0.0, -0.05, 3.0, 1e-6], device="cuda"))
    for causal in (True, False):
        r = _run(fa, c, 0.125, causal, kw)
        _settled(fa)
        _check(c, r, 0.125, causal, kw)


@pytest.mark.parametrize("pre", [0, 1, 127, 128, 129, 255, 256, 300, 383, 384, 400])
def test_prefixes_around_tiles(fa, pre):  # noqa: F811
    c = _inputs([400, 130], 4, 2, 64, BF, 5)
    kw = dict(prefix_lens=torch.tensor([pre, min(pre, 130)], dtype=torch.int32, device="cuda"), softcap=10.0)
    r = _run(fa, c, 0.125, True, kw)
    _settled(fa)
    _check(c, r, 0.125, True, kw)


def test_plain_scores_by_way_of_the_scored_calls(fa):  # noqa: F811
    """No cap, slopes of zero: the plain calls' results within their bounds, and
    within the narrower ones of D = rowsum(P dP); a scored call without any of them is the plain call, bit for bit."""
    c = _inputs([333, 90], 4, 2, 128, BF, 11)
    plain = _run(fa, c, 0.1, True, {})
    kw = dict(slopes=torch.zeros(4, device="cuda"))
    r = _run(fa, c, 0.1, True, kw)
    _settled(fa)
    for res in (plain, r):
        packed_check(c, res, 0.1, True)
    _check(c, r, 0.1, True, kw)
    o, lse = torch.full_like(plain["o"], CANARY), torch.full_like(plain["lse"], CANARY)
    p = lambda t: t.data_ptr()
    st = fa.flash_attn_packed_scored_fwd(p(c["q"]), p(c["k"]), p(c["v"]), p(o), p(lse), p(c["cu"]), 2, 423, 4, 2, 128, None,
                                         0.1, 1, None, None, None, 0, torch.cuda.current_stream().cuda_stream)
    _settled(fa)
    assert st == 0 and torch.equal(_bits(o), _bits(plain["o"])) and torch.equal(_bits(lse), _bits(plain["lse"]))


def test_streams_and_replayed_graphs(fa):  # noqa: F811
    """Two calls at once on two streams, and a captured step replayed after the
    bounds, prefixes and slopes have changed, over a workspace that is overwritten
    in between."""
    cs = [_inputs([333, 90], 4, 2, d, BF, d) for d in (64, 128)]
    kws = [_score_args([333, 90], 4, cap, True, True, 3) for cap in (0.0, 20.0)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [_outputs(c) for c in cs]
    torch.cuda.synchronize()
    for _ in range(3):
        for c, s, o, kw in zip(cs, streams, outs, kws):
            _run(fa, c, 0.1, True, kw, out=o, stream=s)
    _settled(fa)
    for c, o, kw in zip(cs, outs, kws):
        _check(c, o, 0.1, True, kw)
    c, kw = cs[1], kws[1]
    ws = [torch.empty(fa.flash_attn_packed_workspace_size(2, 423, 4, 2, 128, b), dtype=torch.uint8, device="cuda")
          for b in (0, 1)]
    out = _outputs(c)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _run(fa, c, 0.1, True, kw, out=out, ws=ws)
    for i, cu in enumerate(([0, 333, 423], [0, 1, 423], [0, 200, 200], [10, 300, 410])):
        c["cu"].copy_(torch.tensor(cu, dtype=torch.int32))
        kw["prefix_lens"].copy_(torch.tensor([40 * i, 200 - 50 * i], dtype=torch.int32))
        kw["slopes"].mul_(0.5)
        for t in out.values():
            t.fill_(CANARY)
        for w in ws:
            w.fill_(0xFF)
        g.replay()
        _settled(fa)
        _check(c, out, 0.1, True, kw, cu)


@pytest.mark.parametrize("Hq,Hk", [(4, 2), (64, 64)], ids=["few_tiles", "many_tiles"])
@pytest.mark.parametrize("softcap", [0.0, 30.0])
def test_wait_runs_out_and_device_stays_usable(fa, softcap, Hq, Hk):  # noqa: F811
    c = _inputs([700, 300], Hq, Hk, 64, BF, 5)
    kw = _score_args([700, 300], Hq, softcap, True, True, 6)
    r = _run(fa, c, 0.1, True, kw)
    _settled(fa)
    fa.attention_packed_fwd(c["q"], c["k"], c["v"], c["cu"], 0.1, wait_limit_us=20000, test_stall=1, **kw)
    torch.cuda.synchronize()
    st, detail = fa.device_error()
    assert st == 5 and 310 <= detail[1] < 350, detail
    fa.attention_packed_bwd(c["q"], c["k"], c["v"], r["o"], c["do"], r["lse"], c["cu"], 0.1, wait_limit_us=20000,
                            test_stall=1, **kw)
    torch.cuda.synchronize()
    st, detail = fa.device_error()
    assert st == 5 and 350 <= detail[1] < 400, detail
    _again(fa, c, r, 0.1, True, kw)


def test_helpers_refuse_what_does_not_fit(fa):  # noqa: F811
    c = _inputs([20, 5], 4, 2, 64, BF, 7)
    kw = _score_args([20, 5], 4, 10.0, True, True)
    def bad(**more):
        with pytest.raises((ValueError, fa.FlashAttnError)):
            fa.attention_packed_fwd(c["q"], c["k"], c["v"], c["cu"], 0.1, **{**kw, **more})
    bad(softcap=-1.0)
    bad(softcap=float("nan"))
    bad(softcap=5000.0)
    bad(slopes=kw["slopes"].double())
    bad(slopes=kw["slopes"][:3])
    bad(slopes=kw["slopes"].cpu())
    bad(prefix_lens=kw["prefix_lens"].long())
    bad(prefix_lens=kw["prefix_lens"][:1])
    bad(causal=False)
    _settled(fa)


@pytest.mark.parametrize("softcap", [0.0, 40.0])
def test_slopes_over_long_distances(fa, softcap):  # noqa: F811
    """A row's keys differ by thousands in either direction, so that its maximum
    moves from tile to tile, or lies in the first one."""
    c = _inputs([1500, 700], 4, 2, 128, FH, 12)
    kw = dict(softcap=softcap, slopes=torch.tensor([6.0, -6.0, 0.3, -0.3], device="cuda"))
    for causal in (True, False):
        r = _run(fa, c, 0.09, causal, kw)
        _settled(fa)
        _check(c, r, 0.09, causal, kw)


def test_offsets_past_32_bits(fa):  # noqa: F811
    """The sequences are the last rows of tensors of more than 2^31 elements."""
    Hq, Hk, d, T = 64, 2, 128, 263000
    small = _inputs([150, 290], Hq, Hk, d, BF, 13)
    n = 440
    kw = _score_args([150, 290], Hq, 30.0, True, True)
    big = {k: torch.zeros((T,) + small[k].shape[1:], dtype=BF, device="cuda") for k in ("q", "k", "v", "do")}
    for k, x in big.items():
        x[T - n:] = small[k]
    big["cu"] = small["cu"] + (T - n)
    out = dict(o=torch.zeros_like(big["q"]), dq=torch.zeros_like(big["q"]), dk=torch.zeros_like(big["k"]),
               dv=torch.zeros_like(big["k"]), lse=torch.zeros(Hq, T, device="cuda"))
    _run(fa, big, 0.09, True, kw, out=out)
    _settled(fa)
    got = {k: (x[:, T - n:] if k == "lse" else x[T - n:]) for k, x in out.items()}
    _check(small, got, 0.09, True, kw)
    assert not out["o"][:T - n].any() and not out["dq"][:T - n].any() and not out["dk"][:T - n].any()


@pytest.mark.parametrize("dtype", [BF, FH], ids=["bf16", "fp16"])
@pytest.mark.parametrize("softcap,bias", [(0.5, False), (30.0, False), (50.0, False), (0.0, True), (20.0, True)])
def test_a_row_of_one_key_has_its_value(fa, softcap, bias, dtype):  # noqa: F811
    """Its weight is one, whatever the score: O is V, bit for bit."""
    lens = [1, 1, 5, 1, 300, 1]
    for qmul in (1.0, 40.0):
        c = _inputs(lens, 6, 2, 64, dtype, 14, qmul=qmul)
        kw = _score_args(lens, 6, softcap, bias, False)
        r = _run(fa, c, 0.125, True, kw)
        _settled(fa)
        first = c["cu"][:-1].long()
        assert torch.equal(r["o"][first], c["v"][first].repeat_interleave(3, dim=1))
