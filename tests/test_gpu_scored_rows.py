"""What one row of a capped call may do to another, and scores at the ends of the
cap, on the GPU: a NaN stays in the rows that see it, a sequence's bits do not
depend on what lies behind it, gradients keep their size where the cap is
saturated, and O keeps its precision and range whatever the scores and values."""
import numpy as np
import pytest
import torch

from oracle import scored as S
from test_gpu_packed import BF, FH, _bits, _f64, _inputs, _settled, fa  # noqa: F401 (fa: the fixture)
from test_gpu_scored import _check, _run

pytestmark = pytest.mark.gpu


def _slopes(Hq, bias):
    return dict(slopes=torch.tensor([2.0 ** -(h + 2) for h in range(Hq)], device="cuda")) if bias else {}


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("row", [62, 63, 130])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("softcap,qmul", [(5.0, 8.0), (50.0, 1.0)])
def test_a_nan_query_stays_in_its_row(fa, softcap, qmul, bias, row, d):  # noqa: F811
    """Query `row` is NaN: O and dQ of all other rows, and dV of the keys it does
    not see, are those of the formula, as in the calls of plain scores."""
    c = _inputs([200], 2, 2, d, BF, 21, qmul=qmul)
    kw = dict(softcap=softcap, **_slopes(2, bias))
    val, tol = S.packed_attention(_f64(c["q"]), _f64(c["k"]), _f64(c["v"]), _f64(c["do"]), c["bounds"], 0.125, True,
                                  2.0 ** -8, softcap, None if not bias else kw["slopes"].cpu().numpy())
    c["q"][row] = float("nan")
    r = _run(fa, c, 0.125, True, kw)
    plain = _run(fa, c, 0.125, True, {})
    _settled(fa)
    others = np.arange(200) != row
    unseen = np.arange(200) > row
    for name, key, rows in (("O", "o", others), ("dQ", "dq", others), ("dV", "dv", unseen)):
        assert torch.isfinite(plain[key]).cpu().numpy()[rows].all(), name
        off = np.abs(_f64(r[key]) - val[name])[rows] - tol[name][rows]
        assert off.max() <= 0, f"{name}: {off.max():.3g} over its bound"      # (a NaN fails)
    assert torch.isnan(r["o"][row]).all() and torch.isnan(r["dq"][row]).all() and torch.isnan(r["lse"][:, row]).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("causal", [True, False])
def test_gradients_of_a_saturated_cap(fa, causal, bias, d):  # noqa: F811
    """All scores lie 4 to 12 caps from zero, where the cap's slope is 1e-3 to
    1e-10: dQ and dK keep their relative precision."""
    c = _inputs([150, 33], 2, 1, d, BF, 22)
    g = torch.Generator().manual_seed(5)
    sign = 1.0 - 2.0 * torch.randint(0, 2, (183, 1, 1), generator=g)
    size = 0.5 + torch.rand(183, 2, 1, generator=g)
    c["q"] = ((1 + torch.rand(183, 2, d, generator=g)) * size).to(BF).cuda()
    c["k"] = ((1 + 0.75 * torch.rand(183, 1, d, generator=g)) * sign).to(BF).cuda()   # products of 1 to 3 d, of either sign
    cap, scale = 3.0, 12.0 / d
    kw = dict(softcap=cap, **_slopes(2, bias))
    r = _run(fa, c, scale, causal, kw)
    _settled(fa)
    _check(c, r, scale, causal, kw)
    val, tol = S.packed_attention(_f64(c["q"]), _f64(c["k"]), _f64(c["v"]), _f64(c["do"]), c["bounds"], scale, causal,
                                  2.0 ** -8, cap, None if not bias else kw["slopes"].cpu().numpy(), relative_slope=True)
    for name, key in (("dQ", "dq"), ("dK", "dk")):
        off = np.abs(_f64(r[key]) - val[name]) - tol[name]
        assert off.max() <= 0, f"{name}: {off.max():.3g} over its bound, largest value {np.abs(val[name]).max():.3g}"



@pytest.mark.parametrize("dtype", [BF, FH], ids=["bf16", "fp16"])
@pytest.mark.parametrize("Hq,Hk,d", [(4, 2, 64), (4, 2, 128), (3, 3, 64), (64, 16, 128)])
@pytest.mark.parametrize("softcap,bias,causal", [(50.0, False, True), (50.0, False, False), (50.0, True, True), (700.0, False, True)])
def test_bits_do_not_depend_on_what_lies_behind(fa, softcap, bias, causal, Hq, Hk, d, dtype):  # noqa: F811
    """A sequence whose last tile is not full, before one of huge queries, before
    one of ordinary ones, and before rows of no sequence: the same bits."""
    n = 150
    c = _inputs([n, 140], Hq, Hk, d, dtype, 23)
    kw = dict(softcap=softcap, **_slopes(Hq, bias))
    results = []
    for behind in (1.0, 300.0):
        c["q"][n:] = (c["q"][n:].float() * behind).to(dtype)
        for bounds in ([0, n, n + 140], [0, n, n]):
            c["cu"].copy_(torch.tensor(bounds, dtype=torch.int32))
            r = _run(fa, c, d ** -0.5, causal, kw)
            _settled(fa)
            results.append(r)
    for r in results[1:]:     # (two key tiles: dQ's two partial sums are the same in either order)
        for key in ("o", "dq", "dk", "dv"):
            assert torch.equal(_bits(r[key][:n].contiguous()), _bits(results[0][key][:n].contiguous())), key
        assert torch.equal(_bits(r["lse"][:, :n].contiguous()), _bits(results[0]["lse"][:, :n].contiguous()))
    if Hq <= 4:               # alone: the same kernels (with more heads, calls of few tiles share keys out)
        o, lse = fa.attention_packed_fwd(c["q"][:n], c["k"][:n], c["v"][:n], c["cu"][:2].contiguous(), d ** -0.5, causal=causal, **kw)
        _settled(fa)
        assert torch.equal(_bits(o), _bits(results[0]["o"][:n])) and torch.equal(_bits(lse), _bits(results[0]["lse"][:, :n].contiguous()))



@pytest.mark.parametrize("dtype", [BF, FH], ids=["bf16", "fp16"])
@pytest.mark.parametrize("softcap", [30.0, 50.0, 54.0, 80.0])
@pytest.mark.parametrize("d", [64, 128])
def test_a_row_with_one_heavy_key_has_its_value(fa, d, softcap, dtype):  # noqa: F811
    """Sequences of 2 to 16 tokens; the first key's score is 35 to 75 before the cap,
    the others' at most 0, so that their weights together are below 2^-30 even at a cap
    of 30 (27 after it): O is V of the first key, bit for bit. A rounded weight and an
    unrounded sum would be off by half a step."""
    lens = [2, 3, 5, 9, 16, 16, 7, 2, 2, 4] * 3
    c = _inputs(lens, 4, 2, d, dtype, 24)
    first = c["cu"][:-1].long()
    g = torch.Generator().manual_seed(6)
    T = sum(lens)
    q, k = torch.zeros(T, 4, d), torch.zeros(T, 2, d)
    q[:, :, 0] = 5 + torch.randint(0, 64, (T, 4), generator=g) / 16.0          # 5 to 9, exact in either type
    k[:, :, 0] = -torch.rand(T, 2, generator=g)
    k[first.cpu(), :, 0] = 7 + torch.randint(0, 16, (len(lens), 2), generator=g) / 16.0
    c["q"], c["k"] = q.to(dtype).cuda(), k.to(dtype).cuda()
    kw = dict(softcap=softcap)
    r = _run(fa, c, 1.0, True, kw)
    _settled(fa)
    _check(c, r, 1.0, True, kw)
    want = c["v"][torch.repeat_interleave(first, c["cu"].diff())].repeat_interleave(2, dim=1)
    assert torch.equal(r["o"], want)


@pytest.mark.parametrize("softcap,bias", [(50.0, False), (55.0, False), (54.0, True), (300.0, False), (0.0, True)])
@pytest.mark.parametrize("power", [100, 60, -60, -90])
@pytest.mark.parametrize("d", [64, 128])
def test_values_of_all_sizes(fa, d, power, softcap, bias):  # noqa: F811
    """V, dO or both far from 1, beside scores up to the cap: O and the gradients
    scale with them (the bounds do, too)."""
    c = _inputs([300, 5, 130], 4, 2, d, BF, 25, qmul=10.0)
    c["v"] = (c["v"].float() * 2.0 ** power).to(BF)
    if power > 0:
        c["do"] = (c["do"].float() * 2.0 ** -power).to(BF)
    for causal in (True, False):
        kw = dict(softcap=softcap, **_slopes(4, bias))
        r = _run(fa, c, d ** -0.5, causal, kw)
        _settled(fa)
        _check(c, r, d ** -0.5, causal, kw)


@pytest.mark.parametrize("Hq,Hk", [(4, 2), (64, 64)], ids=["few_tiles", "many_tiles"])
@pytest.mark.parametrize("dtype,d", [(BF, 128), (FH, 64)], ids=["bf16", "fp16"])
def test_wait_runs_out_without_slopes(fa, dtype, d, Hq, Hk):  # noqa: F811
    """Capped scores alone: the device stays usable, and the next call's bits are the first's."""
    c = _inputs([700, 300], Hq, Hk, d, dtype, 5)
    kw = dict(softcap=30.0)
    r = _run(fa, c, 0.1, True, kw)
    _settled(fa)
    fa.attention_packed_fwd(c["q"], c["k"], c["v"], c["cu"], 0.1, wait_limit_us=20000, test_stall=1, **kw)
    torch.cuda.synchronize()
    st, detail = fa.device_error()
    assert st == 5 and 310 <= detail[1] < 350, detail
    r2 = _run(fa, c, 0.1, True, kw)
    _settled(fa)
    for key in ("o", "lse", "dk", "dv"):
        assert torch.equal(_bits(r[key].contiguous()), _bits(r2[key].contiguous())), key


@pytest.mark.parametrize("dtype", [BF, FH], ids=["bf16", "fp16"])
@pytest.mark.parametrize("order", ["rising", "falling"])
@pytest.mark.parametrize("softcap,causal,prefix", [(50.0, True, False), (50.0, False, False), (300.0, True, True), (20.0, True, True)])
def test_capped_scores_that_grow_along_the_keys(fa, softcap, causal, prefix, order, dtype):  # noqa: F811
    """Scores from one end of the cap to the other along a sequence, so that rows'
    references move from key tile to key tile, or never."""
    c = _inputs([900, 260], 4, 2, 64, dtype, 26, qmul=4.0)
    T = 1160
    rise = torch.linspace(-1.5, 1.5, T, device="cuda").view(T, 1, 1) * (1 if order == "rising" else -1)
    c["q"], c["k"] = c["q"].abs(), (c["k"].float().abs() * rise).to(dtype)
    kw = dict(softcap=softcap)
    if prefix:
        kw["prefix_lens"] = torch.tensor([500, 260], dtype=torch.int32, device="cuda")
    r = _run(fa, c, 0.2, causal, kw)
    _settled(fa)
    _check(c, r, 0.2, causal, kw)
