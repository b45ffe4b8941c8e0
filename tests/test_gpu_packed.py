"""Attention over packed sequences on the GPU against the float64 reference,
element by element within the bounds that oracle/packed.py derives from the
roundings. Rows of no sequence hold NaN in every input and a canary in every
output."""
import numpy as np
import pytest
import torch

from oracle import cache as C
from oracle.packed import packed_attention

pytestmark = pytest.mark.gpu

BF, FH = torch.bfloat16, torch.float16
CANARY = 77.0


@pytest.fixture(scope="module")
def fa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import exact_io_aware_39_gb300 as pkg
    from exact_io_aware_39_gb300 import build as b
    pkg.load(b.build())
    return pkg


def _settled(fa):
    torch.cuda.synchronize()
    st, detail = fa.device_error()
    assert st == 0, detail


def _bits(t):
    return t.view({2: torch.int16, 4: torch.int32}[t.element_size()])


def _inputs(lens, Hq, Hk, d, dtype, seed=0, before=0, behind=0, fused=False, qmul=1.0):
    cu = [before]
    for n in lens:
        cu.append(cu[-1] + n)
    T = cu[-1] + behind
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, Hq + 2 * Hk, d, generator=g)
    x[:, :Hq] *= qmul
    do = torch.randn(T, Hq, d, generator=g)
    for t in (x, do):
        t[:before] = float("nan")
        t[cu[-1]:] = float("nan")
    x, do = x.to(dtype).cuda(), do.to(dtype).cuda()
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    return dict(q=q, k=k, v=v, do=do, cu=torch.tensor(cu, dtype=torch.int32, device="cuda"), bounds=cu, fused=fused)


def _outputs(c):
    T, Hq, d = c["q"].shape
    Hk, dt = c["k"].shape[1], c["q"].dtype
    full = lambda *s, dtype=dt: torch.full(s, CANARY, dtype=dtype, device="cuda")
    out = dict(o=full(T, Hq, d), lse=full(Hq, T, dtype=torch.float32))
    if c["fused"]:                       # gradients as views of one tensor too
        g = full(T, Hq + 2 * Hk, d)
        out.update(dq=g[:, :Hq], dk=g[:, Hq:Hq + Hk], dv=g[:, Hq + Hk:])
    else:
        out.update(dq=full(T, Hq, d), dk=full(T, Hk, d), dv=full(T, Hk, d))
    return out


def _run(fa, c, scale, causal, out=None, ws=(None, None), **kw):
    r = _outputs(c) if out is None else out
    fa.attention_packed_fwd(c["q"], c["k"], c["v"], c["cu"], scale, causal=causal, out=r["o"], lse=r["lse"],
                            workspace=ws[0], **kw)
    fa.attention_packed_bwd(c["q"], c["k"], c["v"], r["o"], c["do"], r["lse"], c["cu"], scale, causal=causal,
                            dq=r["dq"], dk=r["dk"], dv=r["dv"], workspace=ws[1], **kw)
    return r


def _f64(t):
    return t.float().cpu().double().numpy()


def _check(c, r, scale, causal, bounds=None):
    u = 2.0 ** -8 if c["q"].dtype == BF else 2.0 ** -11
    val, tol = packed_attention(_f64(c["q"]), _f64(c["k"]), _f64(c["v"]), _f64(c["do"]),
                                c["bounds"] if bounds is None else bounds, scale, causal, u)
    for name, key in (("O", "o"), ("LSE", "lse"), ("dQ", "dq"), ("dK", "dk"), ("dV", "dv")):
        got, ref = _f64(r[key]), val[name]
        none = np.isnan(ref)
        assert (got[none] == CANARY).all(), f"{name}: rows of no sequence were written"
        assert np.isfinite(got).all(), f"{name} is not finite"
        over = np.abs(got[~none] - ref[~none]) - tol[name][~none]
        assert over.size == 0 or over.max() <= 0, f"{name}: {over.max():.3g} over its bound"


CASES = [
    # lens, Hq, Hk, d, causal, before, behind, fused
    ([1], 1, 1, 64, True, 0, 0, False), ([128], 2, 2, 128, True, 0, 0, False), ([129], 4, 1, 64, False, 0, 5, True),
    ([127, 1, 128, 256, 0, 3], 4, 2, 128, True, 3, 200, True), ([300, 0, 511], 6, 2, 64, True, 0, 1, False),
    ([640], 3, 1, 128, False, 1, 0, True), ([1000, 24], 5, 1, 64, True, 0, 0, True),
    ([17, 40, 5, 60, 33], 8, 2, 80, False, 0, 130, False), ([250, 390], 4, 4, 40, True, 0, 0, True),
    ([200, 257], 2, 1, 8, True, 7, 9, False), ([383, 385, 2], 8, 1, 120, False, 0, 0, True),
    ([0, 0, 5], 2, 2, 96, True, 0, 0, False), ([70] * 30, 4, 2, 128, False, 0, 0, True),
]


@pytest.mark.parametrize("dtype", [BF, FH], ids=["bf16", "fp16"])
@pytest.mark.parametrize("lens,Hq,Hk,d,causal,before,behind,fused", CASES)
def test_forward_and_gradients(fa, lens, Hq, Hk, d, causal, before, behind, fused, dtype):
    c = _inputs(lens, Hq, Hk, d, dtype, len(lens), before, behind, fused)
    scale = d ** -0.5
    r = _run(fa, c, scale, causal)
    _settled(fa)
    _check(c, r, scale, causal)
    r2 = _run(fa, c, scale, causal)
    _settled(fa)
    for key in ("o", "lse", "dk", "dv"):     # (dQ's partial sums are added as they come)
        assert torch.equal(_bits(r[key].contiguous()), _bits(r2[key].contiguous())), key


@pytest.mark.parametrize("d,causal", [(64, True), (128, False)])
def test_more_sequences_than_a_block_has_threads(fa, d, causal):
    lens = [(5 * b) % 4 for b in range(2500)]
    c = _inputs(lens, 2, 1, d, BF, 1)
    r = _run(fa, c, 0.2, causal)
    _settled(fa)
    _check(c, r, 0.2, causal)


@pytest.mark.parametrize("B", [40, 130])
@pytest.mark.parametrize("Hq,Hk,d,causal", [(2, 2, 64, True), (4, 2, 128, True), (3, 1, 128, False), (4, 1, 64, False)])
def test_many_sequences_of_several_tiles(fa, Hq, Hk, d, causal, B):
    """Lists of more than 32 sequences (several to a lane) and of more than 128
    (made by the plan kernel)."""
    lens = [(97 * b) % 401 for b in range(B)]
    c = _inputs(lens, Hq, Hk, d, BF, 8, 2, 70)
    r = _run(fa, c, d ** -0.5, causal)
    _settled(fa)
    _check(c, r, d ** -0.5, causal)


@pytest.mark.parametrize("B", [31, 32, 33, 127, 128, 129])
def test_either_side_of_the_direct_list(fa, B):
    c = _inputs([(61 * b) % 150 for b in range(B)], 4, 2, 64, BF, 9)
    r = _run(fa, c, 0.125, True)
    _settled(fa)
    _check(c, r, 0.125, True)


@pytest.mark.parametrize("lens,Hq,Hk,causal", [([300, 140, 1000, 128, 1], 12, 3, True), ([1300], 14, 7, True),
                                               ([700, 90, 0, 129], 8, 8, False), ([257, 256, 255], 5, 1, True)])
@pytest.mark.parametrize("d,dtype", [(64, BF), (128, FH), (96, BF)])
def test_query_tiles_on_their_own(fa, lens, Hq, Hk, causal, d, dtype):
    """Few query tiles: the forward takes one to an item, its key tiles in turn
    by two groups, up to two items to a block and items of one key tile between."""
    c = _inputs(lens, Hq, Hk, d, dtype, 15, 2, 9, True)
    T = c["q"].shape[0]
    assert T > 128 * len(lens) and (T // 128 + len(lens)) * Hq <= (256 if causal else 152)
    for qmul in (1.0, 20.0):          # (20: the groups' references differ)
        c["q"].mul_(qmul)
        r = _run(fa, c, d ** -0.5, causal)
        _settled(fa)
        _check(c, r, d ** -0.5, causal)
        r2 = _run(fa, c, d ** -0.5, causal)
        _settled(fa)
        for key in ("o", "lse", "dk", "dv"):
            assert torch.equal(_bits(r[key].contiguous()), _bits(r2[key].contiguous())), key


@pytest.mark.parametrize("Hq,Hk,d,causal,dtype", [(32, 16, 64, True, BF), (16, 16, 128, True, FH),
                                                  (48, 16, 128, False, BF), (16, 16, 40, False, BF)])
def test_items_enough_to_stay_whole(fa, Hq, Hk, d, causal, dtype):
    """More than two items of the backward for every SM: dK and dV are written
    by the items themselves. (The other tests have fewer, whose parts are
    summed.)"""
    lens = [400, 300, 129, 77, 128, 1, 0, 250, 513]
    c = _inputs(lens, Hq, Hk, d, dtype, 13, 3, 5, True)
    assert (c["q"].shape[0] // 128 + len(lens)) * Hk >= 304
    r = _run(fa, c, d ** -0.5, causal)
    _settled(fa)
    _check(c, r, d ** -0.5, causal)
    r2 = _run(fa, c, d ** -0.5, causal)
    _settled(fa)
    for key in ("o", "lse", "dk", "dv"):
        assert torch.equal(_bits(r[key].contiguous()), _bits(r2[key].contiguous())), key


@pytest.mark.parametrize("G,n,causal", [(1, 900, True), (1, 900, False), (7, 260, True), (16, 128, False), (5, 1, True)])
def test_items_in_parts(fa, G, n, causal):
    """One key/value head: an item's steps (query head, query tile) in up to 16
    ranges that begin and end inside a head."""
    c = _inputs([n], G, 1, 64, BF, 14)
    r = _run(fa, c, 0.125, causal)
    _settled(fa)
    _check(c, r, 0.125, causal)


def test_head_major_layout(fa):
    """[heads, tokens, d] tensors seen as [tokens, heads, d]: the head stride is
    the larger one."""
    c = _inputs([200, 131], 4, 2, 64, BF, 10)
    for n in ("q", "k", "v", "do"):
        c[n] = c[n].transpose(0, 1).contiguous().transpose(0, 1)
    out = _outputs(c)
    for n in ("o", "dq", "dk", "dv"):
        out[n] = out[n].transpose(0, 1).contiguous().transpose(0, 1)
    r = _run(fa, c, 0.125, True, out=out)
    _settled(fa)
    _check(c, r, 0.125, True)


@pytest.mark.parametrize("d,causal", [(64, False), (128, True)])
def test_long_sequences(fa, d, causal):
    c = _inputs([2300, 700], 2, 1, d, BF, 2, 0, 30, True)
    r = _run(fa, c, d ** -0.5, causal)
    _settled(fa)
    _check(c, r, d ** -0.5, causal)


@pytest.mark.parametrize("d", [64, 128])
def test_large_scores(fa, d):
    """Scores in the hundreds: the reference maximum moves often."""
    c = _inputs([400, 77], 4, 2, d, BF, 3, qmul=30.0)
    r = _run(fa, c, 0.25, True)
    _settled(fa)
    _check(c, r, 0.25, True)


def test_offsets_past_32_bits(fa):
    """Every tensor a view of one buffer whose tokens are 2^26 elements apart:
    the last tokens lie past 2^31 elements. The results are those of small
    tensors, bit for bit (dQ's sums have one term here)."""
    T, Hq, Hk, d = 40, 4, 2, 64
    c = _inputs([33, 7], Hq, Hk, d, BF, 12)
    want = _run(fa, c, 0.125, True)
    _settled(fa)
    big = torch.empty(T, 1 << 26, dtype=BF, device="cuda")
    at = 1 << 25
    def far(x):
        nonlocal at
        y = big[:, at:at + x.shape[1] * d].view(T, x.shape[1], d)
        at += x.shape[1] * d
        return y.copy_(x)
    f = {n: far(c[n]) for n in ("q", "k", "v", "do")}
    f["cu"] = c["cu"]
    out = {n: far(torch.full_like(t, CANARY)) for n, t in want.items() if n != "lse"}
    out["lse"] = torch.full_like(want["lse"], CANARY)
    _run(fa, f, 0.125, True, out=out)
    _settled(fa)
    for n, t in want.items():
        assert torch.equal(_bits(t), _bits(out[n].contiguous())), n


def test_empty_calls(fa):
    for T, cu in ((0, [0, 0, 0]), (5, [0]), (5, [2, 2, 2])):
        q = torch.randn(T, 4, 64, device="cuda").to(BF)
        k = torch.randn(T, 2, 64, device="cuda").to(BF)
        c = dict(q=q, k=k, v=k.clone(), do=q.clone(), cu=torch.tensor(cu, dtype=torch.int32, device="cuda"), fused=False)
        r = _run(fa, c, 0.1, True)
        _settled(fa)
        for t in r.values():
            assert (t == CANARY).all()


@pytest.mark.parametrize("cu", [[0, 100, 50, 150], [0, 100, 400], [-5, 100, 150], [0, 150, 0, 150, 0, 150],
                                [0, 150] * 25, [0, 150] * 70])
def test_bounds_that_are_no_sequences_are_left_out(fa, cu):
    """Decreasing bounds or bounds outside the tensors: those sequences are left
    out and the error word says so; the others (where they do not overlap)
    are computed."""
    c = _inputs([150], 2, 1, 64, BF, 4)
    c["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    r = _run(fa, c, 0.2, True)
    torch.cuda.synchronize()
    st, detail = fa.device_error()
    assert st == 6 and detail[1] == 300, detail
    if cu[1:3] == [100, 400]:
        _check(c, r, 0.2, True, [0, 100])
    if cu[0] == -5:
        _check(c, r, 0.2, True, [100, 150])
    assert fa.device_error()[0] == 0


def test_streams_and_replayed_graphs(fa):
    """Two calls at once on two streams, and a captured step replayed after the
    bounds have changed, over a workspace that is overwritten in between."""
    cs = [_inputs([333, 90], 4, 2, d, BF, d) for d in (64, 128)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = [_outputs(c) for c in cs]
    torch.cuda.synchronize()
    for _ in range(3):
        for c, s, o in zip(cs, streams, outs):
            _run(fa, c, 0.1, True, out=o, stream=s)
    _settled(fa)
    for c, o in zip(cs, outs):
        _check(c, o, 0.1, True)
    c = cs[1]
    size = lambda b: fa.flash_attn_packed_workspace_size(2, 423, 4, 2, 128, b)
    ws = [torch.empty(size(b), dtype=torch.uint8, device="cuda") for b in (0, 1)]
    out = _outputs(c)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _run(fa, c, 0.1, True, out=out, ws=ws)
    for cu in ([0, 333, 423], [0, 1, 423], [0, 200, 200], [10, 300, 410]):
        c["cu"].copy_(torch.tensor(cu, dtype=torch.int32))
        for t in out.values():
            t.fill_(CANARY)
        for w in ws:
            w.fill_(0xFF)
        g.replay()
        _settled(fa)
        _check(c, out, 0.1, True, cu)


@pytest.mark.parametrize("Hq,Hk", [(4, 2), (64, 64)], ids=["few_tiles", "many_tiles"])
@pytest.mark.parametrize("d", [64, 128])
def test_wait_runs_out_and_device_stays_usable(fa, d, Hq, Hk):
    c = _inputs([700, 300], Hq, Hk, d, BF, 5)
    r = _run(fa, c, 0.1, True)
    _settled(fa)
    fa.attention_packed_fwd(c["q"], c["k"], c["v"], c["cu"], 0.1, wait_limit_us=20000, test_stall=1)
    torch.cuda.synchronize()
    st, detail = fa.device_error()
    assert st == 5 and 310 <= detail[1] < 350, detail
    fa.attention_packed_bwd(c["q"], c["k"], c["v"], r["o"], c["do"], r["lse"], c["cu"], 0.1, wait_limit_us=20000,
                            test_stall=1)
    torch.cuda.synchronize()
    st, detail = fa.device_error()
    assert st == 5 and 350 <= detail[1] < 400, detail
    r2 = _run(fa, c, 0.1, True)
    _settled(fa)
    for key in ("o", "lse", "dk", "dv"):
        assert torch.equal(_bits(r[key]), _bits(r2[key])), key


def test_prompts_then_cache_then_tokens(fa):
    """As a server runs them: prompts through the packed forward, their keys and
    values into the cache, then one token at a time against the cache. Each
    token's output is also the last row of the whole sequence's attention."""
    Hq, Hk, d, page, steps = 8, 2, 64, 16, 3
    lens = [37, 1, 64]
    total = [n + steps for n in lens]
    c = _inputs(total, Hq, Hk, d, BF, 6, fused=True)
    whole = _run(fa, c, 0.125, True)
    _settled(fa)
    for e4m3 in (False, True):
        pages = 16
        mk = lambda: torch.zeros(pages, Hk, page, d, device="cuda").to(torch.float8_e4m3fn if e4m3 else BF)
        sc = (lambda: torch.ones(pages, Hk, page, device="cuda")) if e4m3 else (lambda: None)
        kc, vc, ks, vs = mk(), mk(), sc(), sc()
        need = [-(-n // page) for n in total]
        perm = torch.randperm(pages, generator=torch.Generator().manual_seed(1))
        table = torch.full((3, max(need)), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = perm[at:at + n].int()
            at += n
        slot = lambda b, j: int(table[b, j // page]) * page + j % page
        start = c["bounds"]
        rows = torch.cat([torch.arange(start[b], start[b] + lens[b]) for b in range(3)]).cuda()
        slots = torch.tensor([slot(b, j) for b in range(3) for j in range(lens[b])], device="cuda")
        pc = dict(q=c["q"][rows], k=c["k"][rows], v=c["v"][rows], do=c["do"][rows], fused=False,
                  cu=torch.tensor([0, 37, 38, 102], dtype=torch.int32, device="cuda"))
        o, _ = fa.attention_packed_fwd(pc["q"], pc["k"], pc["v"], pc["cu"], 0.125)
        fa.kv_cache_write(pc["k"], pc["v"], slots, kc, vc, ks, vs)
        _settled(fa)
        assert torch.equal(_bits(o), _bits(whole["o"][rows]))     # a longer sequence's first rows
        for t in range(steps):
            new = torch.tensor([start[b] + lens[b] + t for b in range(3)], device="cuda")
            fa.kv_cache_write(c["k"][new], c["v"][new],
                              torch.tensor([slot(b, lens[b] + t) for b in range(3)], device="cuda"), kc, vc, ks, vs)
            seq = torch.tensor([n + t + 1 for n in lens], dtype=torch.int32, device="cuda")
            o, lse = fa.attention_cached_fwd(c["q"][new][:, None], kc, vc, table.cuda(), seq, 0.125, k_scale=ks, v_scale=vs)
            _settled(fa)
            f = lambda x, s: _f64(x) * (1.0 if s is None else s.cpu().double().numpy()[..., None])
            ro, rl, absv, mag = C.cached_attention(_f64(c["q"][new][:, None]), f(kc, ks), f(vc, vs), table.numpy(),
                                                   seq.cpu().numpy(), 0.125)
            u = 2.0 ** -8
            ds = ((d + 4) * 2.0 ** -24 * mag + 2.0 ** -20).transpose(0, 2, 1)[..., None]
            tol = (u + 2 * ds) * absv + u * np.abs(ro) + 100 * 2.0 ** -25 * np.abs(f(vc, vs)).max()
            assert (np.abs(_f64(o) - ro) <= tol).all()
            if not e4m3:
                # both are within their bounds of the same value: twice the bound apart
                assert (np.abs(_f64(o[:, 0]) - _f64(whole["o"][new])) <= 2 * tol[:, 0]).all()


def test_helpers_refuse_what_does_not_fit(fa):
    c = _inputs([20, 5], 4, 2, 64, BF, 7)
    r = _run(fa, c, 0.1, True)
    _settled(fa)
    q, k, v, cu = c["q"], c["k"], c["v"], c["cu"]
    def bad(f, **kw):
        with pytest.raises((ValueError, fa.FlashAttnError)):
            f(**kw)
    base = dict(q=q, k=k, v=v, cu_seqlens=cu, scale=0.1)
    def fwd(**kw):
        bad(fa.attention_packed_fwd, **{**base, **kw})
    fwd(q=q.float())
    fwd(q=q[None])
    fwd(k=k.half())
    fwd(v=v[:-1])
    fwd(k=k[:, :, :32])
    fwd(q=q[:, :3])
    fwd(q=q.transpose(1, 2).contiguous().transpose(1, 2))
    fwd(k=k[:, :1].expand(-1, 2, -1))
    fwd(cu_seqlens=cu.long())
    fwd(cu_seqlens=cu.cpu())
    fwd(cu_seqlens=cu[::2])
    fwd(scale=0.0)
    fwd(out=q.float())
    fwd(lse=r["lse"].t())
    fwd(lse=r["lse"].double())
    fwd(workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    basb = dict(q=q, k=k, v=v, o=r["o"], do=c["do"], lse=r["lse"], cu_seqlens=cu, scale=0.1)
    def bwd(**kw):
        bad(fa.attention_packed_bwd, **{**basb, **kw})
    bwd(do=c["do"].half())
    bwd(o=r["o"][1:])
    bwd(lse=r["lse"][:, 1:])
    bwd(dq=r["dk"])
    bwd(dk=r["dq"])
    bwd(dv=r["dv"].cpu())
    bwd(workspace=torch.empty(1 << 20, dtype=torch.uint8, device="cuda")[256:][:512])
    _settled(fa)
