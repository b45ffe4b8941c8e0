"""The paged key/value cache on the GPU against the float64 reference: the
writer bit for bit, the attention of the newest tokens within bounds derived
from its roundings.

Bound of O, element by element, with u = half a step of the 16-bit type
(2^-8 bf16, 2^-11 fp16): P is rounded once (u, or 2^-11 with e4m3, where it is
fp16) and O once (u |O|); a score is off by at most
  dS = (d + 4) 2^-24 mag,   mag = max_j scale sum_c |q_c k_c|
(fp32 sums of d exact products, scale and log2 e), and weights by twice that
plus 2^-20 for the exponential, the sums and the joining factors:
  |dO| <= (u_P + 2 (dS + 2^-20)) sum_j P_j |V_j| + u |O|.
With e4m3, weights under 2^-14 of the running maximum are fp16 subnormals, off
by 2^-25 of it: n 2^-25 max |V| in all. LSE: dS + 2^-20 plus 2^-23 |LSE|.
"""
import math

import numpy as np
import pytest
import torch

from oracle import cache as C

pytestmark = pytest.mark.gpu

BF, FH = torch.bfloat16, torch.float16


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


def _f64(t):
    return t.detach().float().cpu().double().numpy() if t.dtype != torch.float32 else t.cpu().double().numpy()


# ---------------------------------------------------------------------------
# writer
# ---------------------------------------------------------------------------

def _rows(T, Hk, d, dtype, seed, fused):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, 3 * Hk, d, generator=g) * torch.exp(3 * torch.randn(T, 3 * Hk, 1, generator=g))
    x = x.to(dtype).cuda()
    if fused:
        return x[:, Hk:2 * Hk], x[:, 2 * Hk:]
    return x[:, Hk:2 * Hk].contiguous(), x[:, 2 * Hk:].contiguous()


def _empty_cache(pages, Hk, page, d, dtype, e4m3):
    g = torch.Generator().manual_seed(99)
    mk = lambda: torch.randn(pages, Hk, page, d, generator=g).cuda().to(torch.float8_e4m3fn if e4m3 else dtype)
    sc = (lambda: torch.full((pages, Hk, page), 7.0, device="cuda")) if e4m3 else (lambda: None)
    return mk(), mk(), sc(), sc()


def _bits(t):
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


WRITES = [
    # T, Hk, d, page, dtype, e4m3, fused
    (1, 1, 8, 16, BF, False, False), (1, 1, 16, 16, BF, True, False), (3, 2, 40, 32, FH, False, True),
    (70, 5, 48, 64, FH, True, True), (257, 8, 128, 16, BF, True, True), (129, 3, 64, 256, BF, True, False),
    (64, 4, 112, 128, FH, True, False), (500, 2, 128, 32, FH, False, True), (33, 7, 80, 64, BF, True, True),
]


@pytest.mark.parametrize("T,Hk,d,page,dtype,e4m3,fused", WRITES)
def test_write_is_exact_and_leaves_the_rest(fa, T, Hk, d, page, dtype, e4m3, fused):
    k, v = _rows(T, Hk, d, dtype, 1, fused)
    pages = T // page + 5
    kc, vc, ks, vs = _empty_cache(pages, Hk, page, d, dtype, e4m3)
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(3))[:T]
    if T > 8:
        slots[1], slots[4], slots[7] = -1, pages * page, -(1 << 40)      # skipped
    before = [None if t is None else t.clone() for t in (kc, vc, ks, vs)]
    fa.kv_cache_write(k, v, slots.cuda(), kc, vc, ks, vs)
    _settled(fa)
    kept = [(t, int(s)) for t, s in enumerate(slots) if 0 <= s < pages * page]
    for x, cache, scale, was, was_s in ((k, kc, ks, before[0], before[2]), (v, vc, vs, before[1], before[3])):
        want = _bits(was).cpu().clone()
        want_s = None if was_s is None else was_s.cpu().clone()
        xs = x.cpu()
        for t, s in kept:
            if e4m3:
                y, sc = C.e4m3_rows(_f64(xs[t]))
                want[s // page, :, s % page] = _bits(torch.from_numpy(y).to(torch.float8_e4m3fn))
                want_s[s // page, :, s % page] = torch.from_numpy(sc).float()
            else:
                want[s // page, :, s % page] = _bits(xs[t])
        assert torch.equal(_bits(cache).cpu(), want)
        if e4m3:
            assert torch.equal(scale.cpu(), want_s)


def test_write_edges_of_the_quantisation(fa):
    """Rows at the edges: zeros, the smallest and largest numbers, maxima at
    and just over 448 2^e, halfway cases, infinities and NaN."""
    d = 16
    rows = []
    for dtype in (BF, FH):
        big, tiny = torch.finfo(dtype).max, torch.finfo(dtype).smallest_normal
        r = torch.zeros(12, d)
        r[1, 3], r[2, :2] = tiny, torch.tensor([big, -tiny])
        r[3, :3] = torch.tensor([448.0, 17.0, 0.017])
        r[4, :3] = torch.tensor([450.0, -449.9, 1.0])        # (448 or 450 in 16 bits)
        r[5] = torch.arange(d) * 1.0625
        r[6, :3] = torch.tensor([float("inf"), -3.0, 2.0])
        r[7, :3] = torch.tensor([float("nan"), -300.0, 0.001])
        r[8] = float("-inf")
        r[9] = 2.0 ** -20 * torch.arange(d)
        r[10] = torch.linspace(-448, 448, d)
        r[11, 0], r[11, 1] = 464.0, 1.8125
        rows.append((dtype, r.to(dtype)))
    for dtype, r in rows:
        k = r[:, None].cuda()
        kc, vc, ks, vs = _empty_cache(1, 1, 16, d, dtype, True)
        fa.kv_cache_write(k, k, torch.arange(12, device="cuda"), kc, vc, ks, vs)
        _settled(fa)
        y, sc = C.e4m3_rows(_f64(r))
        got = kc[0, 0, :12].float().cpu().numpy()
        assert np.array_equal(np.isnan(got), np.isnan(y))
        assert np.array_equal(np.nan_to_num(got), np.nan_to_num(y))
        assert np.array_equal(ks[0, 0, :12].cpu().numpy(), sc)
        assert torch.equal(_bits(kc), _bits(kc)) and torch.equal(ks, vs)


# ---------------------------------------------------------------------------
# attention against the cache
# ---------------------------------------------------------------------------

def _case(B, Nq, Hq, Hk, d, page, lens, dtype, e4m3, seed=0, spare=3, strided=False, qmul=1.0, room=0):
    """A cache whose places behind the sequences' tokens all hold NaN. room: the
    tokens the table has columns for, where that is more than the lengths need
    (a call of few sequences and little room is joined on chip)."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    pages, width = sum(need) + spare, max(1, max(need), room // page) + 1
    perm = torch.randperm(pages, generator=g)
    table = torch.full((B, width), 1 << 30, dtype=torch.int32)      # behind the last page: not read
    owned = torch.zeros(pages, page, dtype=torch.bool)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n].int()
        for i in range(n):
            owned[perm[at + i], :min(page, lens[b] - i * page)] = True
        at += n
    dead = ~owned[:, None].expand(pages, Hk, page)
    out = {}
    for name in ("k", "v"):
        x = torch.randn(pages, Hk, page, d, generator=g)
        if e4m3:
            x = x * torch.exp2(torch.randint(-6, 7, (pages, Hk, page, 1), generator=g).float())
            y, sc = C.e4m3_rows(x.double().numpy())
            pay, sc = torch.from_numpy(y).to(torch.float8_e4m3fn), torch.from_numpy(sc).float()
            if name == "k":
                sc = sc * 2.0 ** -2
            out[name + "_f64"] = pay.double().numpy() * sc.double().numpy()[..., None]
            pay, sc = _bits(pay).clone(), sc.clone()
            pay[dead] = 0x7F                                        # NaN
            sc[dead] = float("nan")
            out[name], out[name + "s"] = pay.view(torch.float8_e4m3fn).cuda(), sc.cuda()
        else:
            x = x.to(dtype)
            out[name + "_f64"] = x.double().numpy()
            x = x.clone()
            x[dead] = float("nan")
            out[name], out[name + "s"] = x.cuda(), None
    wide = torch.randn(B, Nq, Hq + (3 if strided else 0), d, generator=g) * qmul
    wide = wide.to(dtype).cuda()
    out["q"] = wide[:, :, :Hq] if strided else wide
    out["table"], out["lens"] = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    return out


def _run(fa, c, scale, **kw):
    return fa.attention_cached_fwd(c["q"], c["k"], c["v"], c["table"], c["lens"], scale, k_scale=c["ks"], v_scale=c["vs"],
                                   **kw)


def _check(c, scale, o, lse, lens=None):
    q = c["q"]
    B, Nq, Hq, d = q.shape
    lens = c["lens"].cpu().numpy() if lens is None else lens
    ro, rl, absv, mag = C.cached_attention(_f64(q), c["k_f64"], c["v_f64"], c["table"].cpu().numpy(), lens, scale)
    u = 2.0 ** -8 if q.dtype == BF else 2.0 ** -11
    u_p = 2.0 ** -11 if c["ks"] is not None else u
    ds = ((d + 4) * 2.0 ** -24 * mag + 2.0 ** -20).transpose(0, 2, 1)[..., None]
    tol = (u_p + 2 * ds) * absv + u * np.abs(ro)
    if c["ks"] is not None:
        tol = tol + max(int(max(lens)), 1) * 2.0 ** -25 * np.abs(c["v_f64"]).max()
    got = _f64(o)
    assert np.isfinite(got).all()
    bad = np.abs(got - ro) - tol
    assert bad.max() <= 0, f"O off by {np.abs(got - ro).max():.3g}, {bad.max():.3g} over the bound"
    gl = lse.cpu().double().numpy()
    assert np.array_equal(np.isneginf(gl), np.isneginf(rl))
    fin = np.isfinite(rl)
    lt = ds[..., 0].transpose(0, 2, 1) + 2.0 ** -23 * np.abs(np.where(fin, rl, 0))
    assert (np.abs(gl[fin] - rl[fin]) <= lt[fin]).all(), np.abs(gl[fin] - rl[fin]).max()


CASES = [
    # B, Nq, Hq, Hk, d, page, lens
    (1, 1, 1, 1, 64, 16, [1]), (1, 1, 8, 1, 128, 16, [15]), (2, 1, 4, 4, 128, 32, [16, 17]),
    (4, 1, 8, 2, 64, 64, [0, 33, 64, 5]), (3, 2, 12, 4, 128, 16, [1, 2, 47]), (2, 5, 16, 2, 80, 128, [3, 140]),
    (1, 1, 20, 1, 128, 64, [700]), (5, 1, 6, 3, 48, 256, [255, 256, 257, 1, 0]), (1, 3, 21, 3, 16, 32, [95]),
    (2, 1, 32, 8, 128, 16, [1000, 31]), (1, 1, 16, 2, 128, 64, [5000]), (3, 9, 8, 2, 112, 16, [9, 8, 77]),
]


@pytest.mark.parametrize("kind", ["bf16", "fp16", "bf16_e4m3", "fp16_e4m3"])
@pytest.mark.parametrize("room", [0, 1 << 17], ids=["on_chip", "ranges"])
@pytest.mark.parametrize("B,Nq,Hq,Hk,d,page,lens", CASES)
def test_cached_attention(fa, B, Nq, Hq, Hk, d, page, lens, room, kind):
    dtype, e4m3 = (BF if kind.startswith("bf16") else FH), kind.endswith("e4m3")
    c = _case(B, Nq, Hq, Hk, d, page, lens, dtype, e4m3, seed=len(lens) + d, strided=(Hq % 2 == 0), room=room)
    needs = fa.flash_attn_cached_needs_workspace(B, Nq, Hq, Hk, d, page, c["table"].shape[1], int(e4m3))
    assert needs == (1 if room else 0)
    scale = d ** -0.5
    o, lse = _run(fa, c, scale)
    _settled(fa)
    _check(c, scale, o, lse)
    o2, lse2 = _run(fa, c, scale)
    _settled(fa)
    assert torch.equal(_bits(o), _bits(o2)) and torch.equal(_bits(lse), _bits(lse2))


def test_head_dimension_of_8(fa):
    c = _case(2, 1, 4, 2, 8, 16, [40, 3], BF, False)
    o, lse = _run(fa, c, 0.4)
    _settled(fa)
    _check(c, 0.4, o, lse)


@pytest.mark.parametrize("e4m3", [False, True])
def test_many_sequences_of_all_lengths(fa, e4m3):
    """More sequences than threads of a block, lengths from zero on: the ranges
    of the warps cross many sequences."""
    lens = [(7 * b) % 45 for b in range(600)]
    c = _case(600, 1, 4, 2, 64, 16, lens, BF, e4m3)
    o, lse = _run(fa, c, 0.125)
    _settled(fa)
    _check(c, 0.125, o, lse)


@pytest.mark.parametrize("room", [0, 1 << 17], ids=["on_chip", "ranges"])
def test_large_scores_and_scales_far_apart(fa, room):
    """Scores in the hundreds move the running maximum often; value scales
    2^80 apart must not lose a token whose weight is large."""
    c = _case(2, 1, 8, 2, 128, 16, [300, 90], BF, False, qmul=20.0, room=room)
    o, lse = _run(fa, c, 0.3)
    _settled(fa)
    _check(c, 0.3, o, lse)
    c = _case(1, 1, 4, 1, 64, 16, [64], BF, True, qmul=0.01, room=room)
    e = torch.linspace(-50, 30, 64).round()
    c["vs"][:] = float("nan")
    for j in range(64):
        c["vs"][int(c["table"][0, j // 16]), 0, j % 16] = 2.0 ** float(e[j])
    live = torch.nan_to_num(c["vs"]).double().cpu().numpy()
    c["v_f64"] = np.nan_to_num(c["v"].double().cpu().numpy()) * live[..., None]
    # every score about 0 but the first token's, whose value scale is the smallest: with
    # its score at 60 it takes a weight of e^60 against 2^30 scales elsewhere
    o, lse = _run(fa, c, 1.0)
    _settled(fa)
    _check(c, 1.0, o, lse)
    c["ks"][int(c["table"][0, 0]), 0, 0] *= 2.0 ** 14
    c["k_f64"][int(c["table"][0, 0]), 0, 0] *= 2.0 ** 14
    o, lse = _run(fa, c, 1.0)
    _settled(fa)
    _check(c, 1.0, o, lse)


def test_scales_that_are_no_powers_of_two(fa):
    c = _case(2, 1, 8, 2, 128, 32, [100, 37], FH, True)
    for n in ("k", "v"):
        f = torch.rand(c[n + "s"].shape, generator=torch.Generator().manual_seed(5)) + 0.3
        c[n + "_f64"] = c[n + "_f64"] * f.double().numpy()[..., None]
        c[n + "s"] = c[n + "s"] * f.cuda()
    o, lse = _run(fa, c, 0.05)
    _settled(fa)
    # the product of a scale and its factor is rounded once in fp32 (2^-24)
    _check(c, 0.05, o, lse)


def test_pages_outside_the_cache_read_as_zeros(fa):
    """Entries that name no page are coordinates past the tensor map, which the
    copy unit fills with zeros; nothing out of range is addressed."""
    c = _case(2, 1, 4, 2, 64, 16, [60, 40], BF, False)
    c["table"][0, 1], c["table"][1, 0] = -1, 1 << 30
    o, lse = _run(fa, c, 0.2)
    _settled(fa)
    _check(c, 0.2, o, lse)


def test_lengths_are_clamped_to_the_table(fa):
    c = _case(3, 1, 4, 2, 64, 16, [32, 16, 5], BF, False)
    c["table"] = c["table"][:, :2].contiguous()
    c["lens"] = torch.tensor([1000, -7, 5], dtype=torch.int32, device="cuda")
    o, lse = _run(fa, c, 0.2)
    _settled(fa)
    _check(c, 0.2, o, lse)
    assert (o[1] == 0).all() and torch.isneginf(lse[1]).all()


def test_shared_pages(fa):
    """Two sequences whose tables name the same pages."""
    c = _case(2, 1, 4, 2, 64, 16, [48, 48], BF, False)
    c["table"][1, :2] = c["table"][0, :2]
    o, lse = _run(fa, c, 0.2)
    _settled(fa)
    _check(c, 0.2, o, lse)


@pytest.mark.parametrize("e4m3", [False, True])
def test_pages_past_32_bits(fa, e4m3):
    """A cache of more than 2^31 elements whose last pages are written and read:
    what a small cache gives, bit for bit."""
    B, Hq, Hk, d, page, pages = 2, 8, 8, 128, 64, 36000
    lens = [150, 70]
    k, v = _rows(sum(lens), Hk, d, BF, 8, False)
    ids = [[35999, 1, 33000], [35000, 34999, 0]]
    q = torch.randn(B, 1, Hq, d, generator=torch.Generator().manual_seed(2)).to(BF).cuda()
    res = []
    for n, table in ((6, [[0, 1, 2], [3, 4, 5]]), (pages, ids)):
        mk = lambda: torch.empty(n, Hk, page, d, dtype=torch.float8_e4m3fn if e4m3 else BF, device="cuda")
        sc = lambda: torch.empty(n, Hk, page, device="cuda") if e4m3 else None
        cache = (mk(), mk(), sc(), sc())
        slots = [table[b][j // page] * page + j % page for b in range(B) for j in range(lens[b])]
        fa.kv_cache_write(k, v, torch.tensor(slots, device="cuda"), *cache)
        t = torch.tensor(table, dtype=torch.int32, device="cuda")
        res.append(fa.attention_cached_fwd(q, cache[0], cache[1], t, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                           0.1, k_scale=cache[2], v_scale=cache[3]))
        _settled(fa)
        del cache
    for a, b in zip(*res):
        assert torch.equal(_bits(a), _bits(b)) and torch.isfinite(a.float()).all()


@pytest.mark.parametrize("room", [0, 1 << 17], ids=["on_chip", "ranges"])
def test_other_streams_and_replayed_graphs(fa, room):
    """Two calls at once on two streams with workspaces of their own, and a
    captured call replayed after the lengths have changed."""
    cs = [_case(4, 1, 8, 2, 128, 16, [n, 1, 300, 77], BF, e, seed=n, room=room) for n, e in ((500, False), (40, True))]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    res = []
    for _ in range(3):
        res = [_run(fa, c, 0.1, stream=s) for c, s in zip(cs, streams)]
    _settled(fa)
    for c, (o, lse) in zip(cs, res):
        _check(c, 0.1, o, lse)
    c = cs[0]
    ws = torch.empty(fa.flash_attn_cached_workspace_size(4, 1, 8, 2, 128), dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(res[0][0]), torch.empty_like(res[0][1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _run(fa, c, 0.1, out=o, lse=lse, workspace=ws)
    for lens in ([500, 1, 300, 77], [3, 0, 300, 1], [499, 1, 16, 70]):
        c["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        ws.fill_(0xFF)
        g.replay()
        _settled(fa)
        _check(c, 0.1, o, lse, lens)


def test_write_then_read_step_by_step(fa):
    """A sequence grown token by token through the writer, read after each."""
    for e4m3 in (False, True):
        Hk, d, page, n = 2, 64, 16, 37
        k, v = _rows(n, Hk, d, BF, 5, True)
        kc, vc, ks, vs = _empty_cache(5, Hk, page, d, BF, e4m3)
        table = torch.tensor([[3, 1, 4, 0]], dtype=torch.int32)
        g = torch.Generator().manual_seed(1)
        for t in range(n):
            slot = int(table[0, t // page]) * page + t % page
            fa.kv_cache_write(k[t:t + 1], v[t:t + 1], torch.tensor([slot], device="cuda"), kc, vc, ks, vs)
            if t % 9 and t != n - 1:
                continue
            c = dict(q=torch.randn(1, 1, 8, d, generator=g).to(BF).cuda(), k=kc, v=vc, ks=ks, vs=vs, table=table.cuda(),
                     lens=torch.tensor([t + 1], dtype=torch.int32, device="cuda"))
            for name, cache, sc in (("k", kc, ks), ("v", vc, vs)):
                c[name + "_f64"] = _f64(cache) * (1.0 if sc is None else sc.double().cpu().numpy()[..., None])
            o, lse = _run(fa, c, 0.1)
            _settled(fa)
            _check(c, 0.1, o, lse)


@pytest.mark.parametrize("room", [0, 1 << 17], ids=["on_chip", "ranges"])
@pytest.mark.parametrize("e4m3", [False, True])
def test_wait_runs_out_and_device_stays_usable(fa, e4m3, room):
    # (more than one tile of 32 keys for most warps, so that a second one can fail to come)
    c = _case(2, 1, 8, 2, 128, 16, [50000, 30000] if room else [9000, 7000], BF, e4m3, room=room)
    o, lse = _run(fa, c, 0.1)
    _settled(fa)
    _run(fa, c, 0.1, wait_limit_us=20000, test_stall=1)
    torch.cuda.synchronize()
    st, detail = fa.device_error()
    assert st == 5 and detail[1] == 201, detail
    assert fa.device_error()[0] == 0
    o2, lse2 = _run(fa, c, 0.1)
    _settled(fa)
    assert torch.equal(_bits(o), _bits(o2)) and torch.equal(_bits(lse), _bits(lse2))


def test_helpers_refuse_what_does_not_fit(fa):
    c = _case(2, 1, 4, 2, 64, 16, [20, 5], BF, True)
    q, k, v, t, n = (c[x] for x in ("q", "k", "v", "table", "lens"))
    def bad(**kw):
        a = dict(q=q, k_cache=k, v_cache=v, block_table=t, seq_lens=n, scale=0.1, k_scale=c["ks"], v_scale=c["vs"])
        a.update(kw)
        with pytest.raises((ValueError, fa.FlashAttnError)):
            fa.attention_cached_fwd(**a)
    bad(q=q.float())
    bad(q=q.cpu())
    bad(q=q[..., :32])
    bad(q=q[:1])
    bad(k_cache=k.cpu())
    bad(k_cache=k[..., ::2])
    bad(v_cache=v[:1])
    bad(k_scale=None)
    bad(v_scale=c["vs"].half())
    bad(block_table=t.long())
    bad(block_table=t.t())
    bad(seq_lens=n.cpu())
    bad(scale=-1.0)
    bad(out=torch.empty_like(q).float())
    bad(lse=torch.empty(2, 4, 2, device="cuda"))
    bad(workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    x = torch.zeros(3, 2, 64, dtype=BF, device="cuda")
    s = torch.arange(3, device="cuda")
    def badw(**kw):
        a = dict(k=x, v=x, slots=s, k_cache=k, v_cache=v, k_scale=c["ks"], v_scale=c["vs"])
        a.update(kw)
        with pytest.raises((ValueError, fa.FlashAttnError)):
            fa.kv_cache_write(**a)
    badw(k=x.half())
    badw(v=x[:2])
    badw(slots=s.int())
    badw(slots=s[:2])
    badw(k=x[:, :1], v=x[:, :1])
    badw(k=x.transpose(1, 2).contiguous().transpose(1, 2))
    badw(k_scale=None, v_scale=None)
    badw(k_cache=torch.zeros(3, 2, 16, 64, device="cuda"), v_cache=torch.zeros(3, 2, 16, 64, device="cuda"))
    _settled(fa)


def _check_zero_scales(c, scale, o, lse):
    """As _check, for sequences in which values have a scale of 0. Such a key is
    weighed in units of 2^-64, the writer's smallest scale: s - 64, under 128 for
    the scores here, is rounded to within 2^-18 of log2 units, so the weight (of
    a value of zeros, which counts in the sum alone) to within 2^-18 of itself.
    LSE takes that error, and half a step and the error of log2 of a sum of up to
    2^128 in the same units (2^-18 + 2^-17): 2^-16 in all, times ln 2. A weight in
    fp16 is off by up to 2^-25 of the largest, whose key adds 1 / its scale to the
    sum: 2^-25 448 scale a key, and 448 scale is at most twice the row's maximum."""
    q = c["q"]
    ro, rl, absv, mag = C.cached_attention(_f64(q), c["k_f64"], c["v_f64"], c["table"].cpu().numpy(),
                                           c["lens"].cpu().numpy(), scale)
    assert 1.45 * mag.max() < 60                            # |s| in log2 units
    u = 2.0 ** -8 if q.dtype == BF else 2.0 ** -11
    ds = ((q.shape[3] + 4) * 2.0 ** -24 * mag + 2.0 ** -20).transpose(0, 2, 1)[..., None]
    tol = (2.0 ** -11 + 2 * ds + 2.0 ** -17) * absv + u * np.abs(ro)
    tol = tol + 2 * int(c["lens"].max()) * 2.0 ** -25 * np.abs(c["v_f64"]).max()
    got, gl = _f64(o), lse.cpu().double().numpy()
    assert np.isfinite(got).all() and np.isfinite(gl).all()
    assert (np.abs(got - ro) <= tol).all(), np.abs(got - ro).max()
    lt = ds[..., 0].transpose(0, 2, 1) + 2.0 ** -23 * np.abs(rl) + 2.0 ** -16
    assert (np.abs(gl - rl) <= lt).all(), np.abs(gl - rl).max()
    return ro


@pytest.mark.parametrize("dtype", [BF, FH], ids=["bf16", "fp16"])
@pytest.mark.parametrize("room", [0, 1 << 17], ids=["on_chip", "ranges"])
@pytest.mark.parametrize("d,page", [(64, 16), (64, 64), (128, 16), (128, 64), (80, 32), (48, 256)])
def test_e4m3_pages_outside_the_cache_and_scales_of_zero(fa, d, page, room, dtype):
    """In an e4m3 cache a page outside it reads as zeros too (scales among them),
    and so does a row whose stored scale is 0, whatever its payload."""
    lens = [150, 70, 33, 64]
    c = _case(4, 2, 8, 2, d, page, lens, dtype, True, seed=4, qmul=0.02, room=room)
    needs = fa.flash_attn_cached_needs_workspace(4, 2, 8, 2, d, page, c["table"].shape[1], 1)
    assert needs == (1 if room else 0)
    t = c["table"].cpu()
    if page < 150:
        c["table"][0, 1] = -1                               # amid a sequence
    c["table"][1, 0] = 1 << 30                              # its first page
    c["table"][2, :-(-33 // page)] = c["k"].shape[0]        # all of it
    gone = [(0, 0), (0, 7), (0, 149), (3, 31), (3, 32), (3, 63)]
    for b, j in gone:                                       # stored zeros under payloads that are none
        at = (int(t[b, j // page]), slice(None), j % page)
        c["vs"][at] = 0.0
        c["v_f64"][at] = 0.0
    at = (int(t[3, 5 // page]), slice(None), 5 % page)
    c["ks"][at] = 0.0
    c["k_f64"][at] = 0.0
    o, lse = _run(fa, c, 0.2)
    _settled(fa)
    ro = _check_zero_scales(c, 0.2, o, lse)
    assert (ro[2] == 0).all() and (o[2] == 0).all()
    # value scales small enough that a unit scale would outweigh them all
    live = c["vs"] == c["vs"]
    c["vs"][live] *= 2.0 ** -40
    c["v_f64"] *= 2.0 ** -40
    o, lse = _run(fa, c, 0.2, lse=lse)
    _settled(fa)
    if dtype == BF:                                         # (fp16 cannot hold such outputs)
        _check_zero_scales(c, 0.2, o, lse)
    # nothing but scales of zero
    c["vs"][live] = 0.0
    c["v_f64"][:] = 0.0
    o, lse = _run(fa, c, 0.2)
    _settled(fa)
    _check_zero_scales(c, 0.2, o, lse)
    assert (o == 0).all()


def test_write_edges_of_the_values(fa):
    """The rows of test_write_edges_of_the_quantisation's kinds as values under
    other keys: each tensor's payloads and scales are its own."""
    d = 32
    for dtype in (BF, FH):
        big, tiny = torch.finfo(dtype).max, torch.finfo(dtype).smallest_normal
        r = torch.zeros(10, d)
        r[1, 30], r[2, 14:18] = -tiny, torch.tensor([big, -tiny, -big, 1.0])
        r[3, 15:19] = torch.tensor([448.0, 17.0, -0.017, 19.0])
        r[4, :3] = torch.tensor([450.0, -449.9, 1.0])
        r[5] = torch.arange(d) * -1.0625
        r[6, 15:18] = torch.tensor([float("-inf"), -3.0, 2.0])
        r[7, 15:18] = torch.tensor([-300.0, float("nan"), 0.001])
        r[8] = float("inf")
        r[9] = torch.linspace(-448, 448, d)
        k, v = r.to(dtype), r.roll(3, 0).flip(1).to(dtype)
        kc, vc, ks, vs = _empty_cache(1, 1, 16, d, dtype, True)
        fa.kv_cache_write(k[:, None].cuda(), v[:, None].cuda(), torch.arange(10, device="cuda"), kc, vc, ks, vs)
        _settled(fa)
        for x, cache, scale in ((k, kc, ks), (v, vc, vs)):
            y, sc = C.e4m3_rows(_f64(x))
            got = cache[0, 0, :10].float().cpu().numpy()
            assert np.array_equal(np.isnan(got), np.isnan(y))
            assert np.array_equal(np.nan_to_num(got), np.nan_to_num(y))
            assert np.array_equal(scale[0, 0, :10].cpu().numpy(), sc)
            assert (scale[0, 0, 10:] == 7.0).all()
