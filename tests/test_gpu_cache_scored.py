"""The paged cache with capped and biased scores on the GPU against the float64
reference: attention of the newest tokens, what each cached token received, and
the cache's shortening.

Bounds, element by element, with u = half a step of the 16-bit type and e_j the
bound of a weight's relative error (oracle/scored.py): P is rounded once (u, or
2^-11 with e4m3, where it is fp16) and O once,
  |dO| <= u_P sum_j P_j |V_j| + sum_j P_j e_j |V_j| + u |O| (+ 2^-25 for fp16,
          whose smallest numbers are multiples of 2^-24),
with e4m3 n 2^-25 max |V| more, for weights that are fp16 subnormals.
LSE: the average of e, 2^-20 and 2^-22 |LSE|. Received weights: the sum of the
terms' errors, and 2^-24 for each addition."""
import numpy as np
import pytest
import torch

from oracle import scored as S
from test_gpu_cache import BF, FH, _bits, _case, _f64, _settled, fa  # noqa: F401 (fa: the fixture)

pytestmark = pytest.mark.gpu


def _host(x):
    return None if x is None else x.double().cpu().numpy()


def _kw(Hq, softcap, bias, seed=0):
    kw = dict(softcap=softcap)
    if bias:
        kw["slopes"] = torch.tensor(2.0 ** -np.random.default_rng(seed).uniform(0, 8, Hq), dtype=torch.float32, device="cuda")
    return kw


def _run(fa, c, scale, kw, **more):  # noqa: F811
    return fa.attention_cached_fwd(c["q"], c["k"], c["v"], c["table"], c["lens"], scale, k_scale=c["ks"], v_scale=c["vs"],
                                   **kw, **more)


def _ref(c, scale, kw, lens=None, lse=None):
    return S.cached_attention(_f64(c["q"]), c["k_f64"], c["v_f64"], c["table"].cpu().numpy(),
                              c["lens"].cpu().numpy() if lens is None else lens, scale, kw.get("softcap", 0.0),
                              _host(kw.get("slopes")), None if lse is None else lse.cpu().numpy())


def _check(c, scale, kw, o, lse, lens=None):
    r = _ref(c, scale, kw, lens)
    u = 2.0 ** -8 if c["q"].dtype == BF else 2.0 ** -11
    tol = (2.0 ** -11 if c["ks"] is not None else u) * r["absv"] + r["errv"] + u * np.abs(r["O"])
    tol += 2.0 ** -25 if c["q"].dtype == FH else 0.0
    if c["ks"] is not None:
        tol += int(c["lens"].max()) * 2.0 ** -25 * np.abs(c["v_f64"]).max()
    got = _f64(o)
    assert np.isfinite(got).all()
    bad = np.abs(got - r["O"]) - tol
    assert bad.max() <= 0, f"O off by {np.abs(got - r['O']).max():.3g}, {bad.max():.3g} over the bound"
    gl, rl = lse.cpu().double().numpy(), r["LSE"]
    assert np.array_equal(np.isneginf(gl), np.isneginf(rl))
    fin = np.isfinite(rl)
    lt = np.expm1(r["avg"]) + 2.0 ** -20 + 2.0 ** -22 * np.abs(np.where(fin, rl, 0))
    assert (np.abs(gl[fin] - rl[fin]) <= lt[fin]).all(), np.abs(gl[fin] - rl[fin]).max()


SHAPES = [
    # B, Nq, Hq, Hk, d, page, lens
    (1, 1, 1, 1, 64, 16, [1]), (1, 1, 8, 1, 128, 16, [15]), (2, 1, 4, 4, 128, 32, [16, 17]),
    (4, 1, 8, 2, 64, 64, [0, 33, 64, 5]), (3, 2, 12, 4, 128, 16, [1, 2, 47]), (2, 5, 16, 2, 80, 128, [3, 140]),
    (5, 1, 6, 3, 48, 256, [255, 256, 257, 1, 0]), (1, 3, 21, 3, 16, 32, [95]), (2, 1, 32, 8, 128, 16, [1000, 31]),
    (1, 40, 8, 2, 128, 64, [700]), (3, 9, 8, 2, 112, 16, [9, 8, 77]),
]
SCORES = [(30.0, False, 1.0), (0.0, True, 1.0), (5.0, True, 8.0)]


@pytest.mark.parametrize("kind", ["bf16", "fp16", "bf16_e4m3", "fp16_e4m3"])
@pytest.mark.parametrize("room", [0, 1 << 17], ids=["on_chip", "ranges"])
@pytest.mark.parametrize("softcap,bias,qmul", SCORES)
@pytest.mark.parametrize("B,Nq,Hq,Hk,d,page,lens", SHAPES)
def test_cached_attention(fa, B, Nq, Hq, Hk, d, page, lens, softcap, bias, qmul, room, kind):  # noqa: F811
    dtype, e4m3 = (BF if kind.startswith("bf16") else FH), kind.endswith("e4m3")
    c = _case(B, Nq, Hq, Hk, d, page, lens, dtype, e4m3, seed=len(lens) + d, strided=(Hq % 2 == 0), room=room, qmul=qmul)
    kw = _kw(Hq, softcap, bias)
    o, lse = _run(fa, c, d ** -0.5, kw)
    _settled(fa)
    _check(c, d ** -0.5, kw, o, lse)
    o2, lse2 = _run(fa, c, d ** -0.5, kw)
    _settled(fa)
    assert torch.equal(_bits(o), _bits(o2)) and torch.equal(_bits(lse), _bits(lse2))


@pytest.mark.parametrize("softcap,scale,qmul", [(2.0 ** -10, 0.1, 1.0), (0.5, 0.1, 1.0), (1024.0, 0.1, 300.0), (20.0, 50.0, 10.0)])
def test_caps_of_all_sizes(fa, softcap, scale, qmul):  # noqa: F811
    c = _case(2, 1, 8, 2, 64, 16, [300, 90], FH, False, qmul=qmul)
    o, lse = _run(fa, c, scale, dict(softcap=softcap))
    _settled(fa)
    _check(c, scale, dict(softcap=softcap), o, lse)


# ---------------------------------------------------------------------------
# what each token received
# ---------------------------------------------------------------------------

def _received(fa, c, scale, kw, lse, past, out, **more):  # noqa: F811
    return fa.attention_cached_weights(c["q"], c["k"], c["table"], c["lens"], lse, scale, out, k_scale=c["ks"], past=past,
                                       **kw, **more)


def _check_received(c, scale, kw, lse, past, got, lens=None):
    """Against the reference by the LSE that the call was given; places of no
    token hold what they held (7)."""
    r = _ref(c, scale, kw, lens, lse)
    table, Nq = c["table"].cpu().numpy(), c["q"].shape[1]
    G = c["q"].shape[2] // got.shape[1]
    # The rows are added to the past in blocks of 128: each block is one fp32 addition,
    # off by at most 2^-24 of its result, past + what was received so far. The part of
    # what was received is in tolW's Nq G + 2 roundings, that of the past is here. Each
    # of the Nq G weights counts as 0 below 2^-126, fp32's smallest normal number.
    adds = (Nq * G + 127) // 128
    got, past = _host(got), _host(past)
    page = got.shape[2]
    want, tol = np.full(got.shape, 7.0), np.zeros(got.shape)
    for b, (W, tW) in enumerate(zip(r["W"], r["tolW"])):
        n = W.shape[1]
        for j in range(n):
            p = int(table[b, j // page])
            if not 0 <= p < got.shape[0]:
                continue
            old = past[p, :, j % page] if past is not None and j < n - Nq else 0.0
            want[p, :, j % page] = W[:, j] + old
            tol[p, :, j % page] = tW[:, j] + adds * 2.0 ** -24 * np.abs(old) + Nq * G * 2.0 ** -126
    bad = np.abs(got - want) - tol
    assert bad.max() <= 0, f"off by {np.abs(got - want).max():.3g}, {bad.max():.3g} over the bound"


@pytest.mark.parametrize("kind", ["bf16", "fp16", "bf16_e4m3", "fp16_e4m3"])
@pytest.mark.parametrize("softcap,bias,qmul", SCORES + [(0.0, False, 3.0)])
@pytest.mark.parametrize("B,Nq,Hq,Hk,d,page,lens", SHAPES)
def test_received_weights(fa, B, Nq, Hq, Hk, d, page, lens, softcap, bias, qmul, kind):  # noqa: F811
    dtype, e4m3 = (BF if kind.startswith("bf16") else FH), kind.endswith("e4m3")
    c = _case(B, Nq, Hq, Hk, d, page, lens, dtype, e4m3, seed=len(lens) + d, strided=(Hq % 2 == 0), qmul=qmul)
    kw = _kw(Hq, softcap, bias)
    _, lse = _run(fa, c, d ** -0.5, kw)
    shape = c["k"].shape[:3]
    past = torch.rand(shape, generator=torch.Generator().manual_seed(1)).cuda() * 3
    for given in (None, past):
        got = _received(fa, c, d ** -0.5, kw, lse, given, torch.full(shape, 7.0, device="cuda"))
        _settled(fa)
        _check_received(c, d ** -0.5, kw, lse, given, got)
    again = past.clone()                     # onto itself: the same, where there are tokens
    _received(fa, c, d ** -0.5, kw, lse, again, again)
    _settled(fa)
    at = got != 7.0
    assert torch.equal(again[at], got[at]) and torch.equal(again[~at], past[~at])


@pytest.mark.parametrize("Nq", [1, 4, 20])
@pytest.mark.parametrize("kind", ["bf16", "fp16_e4m3"])
@pytest.mark.parametrize("softcap", [0.0, 12.0])
def test_slopes_of_any_sign(fa, softcap, kind, Nq):  # noqa: F811
    dtype = BF if kind == "bf16" else FH
    for room in (0, 1 << 17):
        c = _case(3, Nq, 4, 2, 128, 32, [2500, 900, 40], dtype, kind.endswith("e4m3"), seed=4, room=room)
        kw = dict(softcap=softcap, slopes=torch.tensor([0.0, -0.05, 4.0, -4.0], device="cuda"))
        o, lse = _run(fa, c, 0.1, kw)
        _settled(fa)
        _check(c, 0.1, kw, o, lse)
        got = _received(fa, c, 0.1, kw, lse, None, torch.full(c["k"].shape[:3], 7.0, device="cuda"))
        _settled(fa)
        _check_received(c, 0.1, kw, lse, None, got)


@pytest.mark.parametrize("Nq", [1, 9])
@pytest.mark.parametrize("e4m3", [False, True])
def test_pages_past_32_bits(fa, e4m3, Nq):  # noqa: F811
    """The last pages of caches of more than 2^31 elements (e4m3: bytes), and the
    same tokens in small caches: the same bits."""
    c = _case(2, Nq, 16, 8, 128, 64, [300, 130], BF, e4m3, spare=0)
    n, pages = c["k"].shape[0], 36000
    big = dict(c)
    for name in ("k", "v", "ks", "vs"):
        if c[name] is not None:
            big[name] = torch.empty((pages,) + c[name].shape[1:], dtype=c[name].dtype, device="cuda")
            _bits(big[name]).zero_()[pages - n:] = _bits(c[name])
    big["table"] = torch.where(c["table"] < n, c["table"] + (pages - n), c["table"])
    kw = _kw(16, 20.0, True)
    (o, lse), (o2, lse2) = _run(fa, c, 0.1, kw), _run(fa, big, 0.1, kw)
    past = torch.rand(c["k"].shape[:3], device="cuda")
    w = _received(fa, c, 0.1, kw, lse, past, torch.full(past.shape, 7.0, device="cuda"))
    past2 = torch.zeros((pages,) + past.shape[1:], device="cuda")
    past2[pages - n:] = past
    w2 = _received(fa, big, 0.1, kw, lse, past2, torch.full(past2.shape, 7.0, device="cuda"))
    _settled(fa)
    assert torch.equal(_bits(o), _bits(o2)) and torch.equal(_bits(lse), _bits(lse2))
    assert torch.equal(w2[pages - n:], w) and bool((w2[:pages - n] == 7.0).all())


@pytest.mark.parametrize("e4m3", [False, True])
def test_received_of_many_sequences(fa, e4m3):  # noqa: F811
    """More sequences than threads of a block, many without a token. The weights
    of a query's keys sum to one."""
    lens = [max(0, (7 * b) % 45 - 6) for b in range(600)]
    c = _case(600, 1, 4, 2, 64, 16, lens, BF, e4m3)
    _, lse = _run(fa, c, 0.125, {})
    got = _received(fa, c, 0.125, {}, lse, None, torch.full(c["k"].shape[:3], 7.0, device="cuda"))
    _settled(fa)
    _check_received(c, 0.125, {}, lse, None, got)
    assert abs(float(got[got != 7.0].sum()) - 4 * sum(n > 0 for n in lens)) < 1e-3


def test_received_from_tokens_that_see_nothing_and_pages_outside(fa):  # noqa: F811
    c = _case(2, 6, 4, 2, 64, 16, [4, 60], BF, False)
    c["table"][1, 1] = -1
    c["table"][1, 3] = c["k"].shape[0]
    _, lse = _run(fa, c, 0.2, {})
    assert torch.isneginf(lse[0, :, :2]).all()
    got = _received(fa, c, 0.2, {}, lse, None, torch.full(c["k"].shape[:3], 7.0, device="cuda"))
    _settled(fa)
    _check_received(c, 0.2, {}, lse, None, got)
    c["lens"] = torch.tensor([-3, 10 ** 6], dtype=torch.int32, device="cuda")   # clamped to the table
    c["table"] = c["table"][:, :3].contiguous()
    c["table"][0] = -1
    _, lse = _run(fa, c, 0.2, {})
    got = _received(fa, c, 0.2, {}, lse, None, torch.full(c["k"].shape[:3], 7.0, device="cuda"))
    _settled(fa)
    _check_received(c, 0.2, {}, lse, None, got)


def test_received_on_streams_and_in_replayed_graphs(fa):  # noqa: F811
    cs = [_case(4, 2, 8, 2, 128, 16, [n, 1, 300, 77], BF, e, seed=n) for n, e in ((500, False), (40, True))]
    kw = _kw(8, 20.0, True)
    lses = [_run(fa, c, 0.1, kw)[1] for c in cs]
    outs = [torch.full(c["k"].shape[:3], 7.0, device="cuda") for c in cs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for c, s, l, o in zip(cs, streams, lses, outs):
            _received(fa, c, 0.1, kw, l, None, o, stream=s)
    _settled(fa)
    for c, l, o in zip(cs, lses, outs):
        _check_received(c, 0.1, kw, l, None, o)
    c = cs[0]
    ws = torch.empty(fa.flash_attn_cached_workspace_size(4, 2, 8, 2, 128), dtype=torch.uint8, device="cuda")
    o, lse, w = torch.empty_like(c["q"]), torch.empty_like(lses[0]), outs[0]
    past = torch.rand_like(w)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _run(fa, c, 0.1, kw, out=o, lse=lse, workspace=ws)
        _received(fa, c, 0.1, kw, lse, past, w)
    for lens in ([500, 1, 300, 77], [3, 0, 300, 1], [0, 0, 0, 0], [499, 1, 16, 70]):
        c["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        w.fill_(7.0)
        g.replay()
        _settled(fa)
        _check(c, 0.1, kw, o, lse, lens)
        _check_received(c, 0.1, kw, lse, past, w, lens)


@pytest.mark.parametrize("e4m3", [False, True])
def test_received_of_many_sequences_and_rows(fa, e4m3):  # noqa: F811
    """As above, with the kernel of many rows: a range has many sequences of one tile."""
    lens = [max(0, (7 * b) % 45 - 6) for b in range(1500)]
    c = _case(1500, 5, 8, 2, 64, 16, lens, BF, e4m3)
    _, lse = _run(fa, c, 0.125, {})
    got = _received(fa, c, 0.125, {}, lse, None, torch.full(c["k"].shape[:3], 7.0, device="cuda"))
    _settled(fa)
    _check_received(c, 0.125, {}, lse, None, got)
    rows = 8 * sum(min(n, 5) for n in lens)   # (tokens before the first see nothing)
    assert abs(float(got[got != 7.0].double().sum()) - rows) < 1e-5 * rows


@pytest.mark.parametrize("kind", ["bf16", "bf16_e4m3", "fp16_e4m3"])
@pytest.mark.parametrize("spread", [3, 15])
@pytest.mark.parametrize("softcap,bias", [(0.0, False), (15.0, True)])
def test_received_by_rows_of_all_sizes(fa, softcap, bias, spread, kind):  # noqa: F811
    """Queries of up to 2^spread times one another's size, some of them zeros."""
    dtype = BF if kind.startswith("bf16") else FH
    c = _case(3, 45, 8, 2, 128, 64, [700, 50, 20], dtype, kind.endswith("e4m3"))
    g = torch.Generator().manual_seed(3)
    size = torch.exp2(-torch.randint(0, spread + 1, (3, 45, 8, 1), generator=g).float())
    size[:, 7] = 0.0
    c["q"] = (c["q"].cpu() * size.to(dtype)).cuda()
    kw = _kw(8, softcap, bias)
    _, lse = _run(fa, c, 0.2, kw)
    past = torch.rand(c["k"].shape[:3], device="cuda")
    got = _received(fa, c, 0.2, kw, lse, past, torch.full(c["k"].shape[:3], 7.0, device="cuda"))
    _settled(fa)
    _check_received(c, 0.2, kw, lse, past, got)


@pytest.mark.parametrize("Nq", [1, 5])
def test_received_by_a_key_with_an_infinite_element(fa, Nq):  # noqa: F811
    """Its scores are -inf: it receives nothing, the others what they did."""
    c = _case(1, Nq, 4, 1, 64, 16, [40], BF, False)
    c["q"][..., 0] = -1.0
    page, at = int(c["table"][0, 1]), 3
    c["k"][page, 0, at, 0] = float("inf")
    _, lse = _run(fa, c, 0.2, {})
    got = _received(fa, c, 0.2, {}, lse, None, torch.full(c["k"].shape[:3], 7.0, device="cuda"))
    _settled(fa)
    assert float(got[page, 0, at]) == 0.0
    assert abs(float(got[got != 7.0].sum()) - 4 * Nq) < 1e-4


@pytest.mark.parametrize("e4m3", [False, True])
def test_wait_of_many_rows_runs_out(fa, e4m3):  # noqa: F811
    c = _case(2, 40, 8, 2, 128, 16, [90000, 70000], BF, e4m3)
    _, lse = _run(fa, c, 0.1, {})
    w = [torch.zeros(c["k"].shape[:3], device="cuda") for _ in range(2)]
    _received(fa, c, 0.1, {}, lse, None, w[0])
    _settled(fa)
    _received(fa, c, 0.1, {}, lse, None, w[1], wait_limit_us=20000, test_stall=1)
    torch.cuda.synchronize()
    st, detail = fa.device_error()
    assert st == 5 and 213 <= detail[1] <= 218, detail
    _received(fa, c, 0.1, {}, lse, None, w[1])
    _settled(fa)
    assert torch.equal(_bits(w[0]), _bits(w[1]))


@pytest.mark.parametrize("e4m3", [False, True])
def test_wait_runs_out_and_device_stays_usable(fa, e4m3):  # noqa: F811
    c = _case(2, 1, 8, 2, 128, 16, [90000, 70000], BF, e4m3)
    _, lse = _run(fa, c, 0.1, {})
    w = [torch.zeros(c["k"].shape[:3], device="cuda") for _ in range(2)]
    _received(fa, c, 0.1, {}, lse, None, w[0])
    _settled(fa)
    _received(fa, c, 0.1, {}, lse, None, w[1], wait_limit_us=20000, test_stall=1)
    torch.cuda.synchronize()
    st, detail = fa.device_error()
    assert st == 5 and detail[1] == 211, detail
    _received(fa, c, 0.1, {}, lse, None, w[1])
    _settled(fa)
    assert torch.equal(_bits(w[0]), _bits(w[1]))


# ---------------------------------------------------------------------------
# the cache's shortening
# ---------------------------------------------------------------------------

def _evict_case(lens, Hk, d, page, dtype, e4m3, budget, ties=False, seed=0):
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    new = [-(-min(max(n, 0), budget) // page) for n in lens]
    pages = sum(need) + sum(new) + 2
    perm = torch.randperm(pages, generator=g).int()
    t, nt = torch.full((len(lens), max(1, *need) + 1), -1).int(), torch.full((len(lens), -(-budget // page)), -1).int()
    at = 0
    for table, counts in ((t, need), (nt, new)):
        for b, n in enumerate(counts):
            table[b, :n] = perm[at:at + n]
            at += n
    rows = lambda: torch.randint(0, 256, (pages, Hk, page, d * (1 if e4m3 else 2)), generator=g, dtype=torch.int32).to(
        torch.uint8).cuda().view(torch.float8_e4m3fn if e4m3 else dtype)
    w = torch.exp(2 * torch.randn(pages, Hk, page, generator=g)) * (torch.rand(pages, Hk, page, generator=g) > 0.2)
    if ties:
        w = (w * 2).round() / 2
    sc = lambda: torch.rand(pages, Hk, page, generator=g).cuda() if e4m3 else None
    return dict(k=rows(), v=rows(), ks=sc(), vs=sc(), w=w.cuda(), table=t.cuda(), new=nt.cuda(),
                lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), page=page)


def _evict(fa, c, budget, recent, **kw):  # noqa: F811
    return fa.kv_cache_evict(c["k"], c["v"], c["w"], c["table"], c["lens"], c["new"], budget, recent, k_scale=c["ks"],
                             v_scale=c["vs"], **kw)


def _check_evict(c, before, new_lens, kept, budget, recent, lens=None):
    """Bit for bit, every place of the caches."""
    lens = c["lens"].tolist() if lens is None else lens
    table, new, page = c["table"].cpu().numpy(), c["new"].cpu().numpy(), c["page"]
    pages, Hk = c["w"].shape[:2]
    stay = S.evict(_host(before["w"]), table, lens, budget, recent, page)
    cap = table.shape[1] * page
    assert new_lens.tolist() == [min(max(n, 0), cap, budget) for n in lens]
    want_kept = np.full((len(lens), Hk, budget), -1)
    names = [n for n in ("k", "v", "ks", "vs", "w") if c[n] is not None]
    bits = lambda x: x.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[x.element_size()]).cpu().numpy()
    was = {n: bits(before[n]) for n in names}
    want = {n: x.copy() for n, x in was.items()}
    for b, heads in enumerate(stay):
        for h, tokens in enumerate(heads):
            want_kept[b, h, :len(tokens)] = tokens
            for i, j in enumerate(tokens):
                src, dst = int(table[b, j // page]), int(new[b, i // page])
                if 0 <= dst < pages:
                    for n in names:
                        want[n][dst, h, i % page] = was[n][src, h, j % page] if 0 <= src < pages else 0
    assert np.array_equal(kept.cpu().numpy(), want_kept)
    for n in names:
        assert np.array_equal(bits(c[n]), want[n]), n


EVICTS = [
    # lens, Hk, d, page, dtype, e4m3, budget, recent, ties
    ([1], 1, 8, 16, BF, False, 1, 0, False), ([2, 0], 1, 16, 16, BF, True, 1, 1, False),
    ([100, 7, 0, 64, 65], 2, 64, 16, FH, False, 64, 16, True), ([300, 299], 3, 128, 64, BF, False, 100, 0, False),
    ([300, 299], 3, 128, 64, BF, True, 100, 100, True), ([1023, 1024, 1025, 1026], 2, 48, 32, FH, True, 1024, 5, True),
    ([2500, 40], 8, 128, 128, BF, False, 37, 8, False), ([5000], 2, 80, 256, BF, False, 4999, 1, True),
    ([70] * 40, 4, 120, 16, FH, False, 33, 2, True),
]


@pytest.mark.parametrize("lens,Hk,d,page,dtype,e4m3,budget,recent,ties", EVICTS)
def test_evict(fa, lens, Hk, d, page, dtype, e4m3, budget, recent, ties):  # noqa: F811
    c = _evict_case(lens, Hk, d, page, dtype, e4m3, budget, ties, seed=budget)
    before = {n: None if x is None or n == "page" else x.clone() for n, x in c.items() if n != "page"}
    new_lens, kept = _evict(fa, c, budget, recent)
    _settled(fa)
    _check_evict(c, before, new_lens, kept, budget, recent)


def test_evict_weights_of_all_kinds(fa):  # noqa: F811
    """Infinities, NaN, negative weights, zeros of both signs, subnormals, and
    all weights the same."""
    c = _evict_case([200, 150, 90], 2, 32, 16, BF, False, 60, seed=3)
    g = torch.Generator().manual_seed(4)
    odd = torch.tensor([float("inf"), float("nan"), -1.0, -float("inf"), 0.0, -0.0, 1e-42, 3e-40, 1.0])
    c["w"] = odd[torch.randint(0, 9, c["w"].shape, generator=g)].cuda()
    c["w"][c["table"][2, :6].long()] = 2.5
    before = {n: None if x is None else x.clone() for n, x in c.items() if n != "page"}
    new_lens, kept = _evict(fa, c, 60, 7)
    _settled(fa)
    _check_evict(c, before, new_lens, kept, 60, 7)
    assert kept[2, 0].tolist() == list(range(53)) + list(range(83, 90))


def test_evict_pages_outside_and_lengths_in_place(fa):  # noqa: F811
    """Old pages outside the cache read as zeros, new ones are not written, lengths
    are clamped to the table; new_lens may be seq_lens."""
    c = _evict_case([100, 60, 40], 2, 64, 16, FH, True, 48, seed=5)
    c["table"][0, 1], c["table"][0, 5] = -1, 1 << 30
    c["new"][1, 1] = -7
    lens = [100, 10 ** 6, -4]
    c["table"] = c["table"][:, :7].contiguous()
    c["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
    before = {n: None if x is None else x.clone() for n, x in c.items() if n != "page"}
    new_lens, kept = _evict(fa, c, 48, 20, new_lens=c["lens"])
    _settled(fa)
    assert new_lens is c["lens"]
    _check_evict(c, before, new_lens, kept, 48, 20, lens)


def test_evict_of_a_long_sequence(fa):  # noqa: F811
    c = _evict_case([40000, 33000], 1, 16, 64, BF, False, 20000, True, seed=6)
    before = {n: None if x is None else x.clone() for n, x in c.items() if n != "page"}
    new_lens, kept = _evict(fa, c, 20000, 1000)
    _settled(fa)
    _check_evict(c, before, new_lens, kept, 20000, 1000)


@pytest.mark.parametrize("lens", [[170000, 3000], [350000]])
def test_evict_of_sequences_that_many_blocks_share(fa, lens):  # noqa: F811
    """More weights than four blocks (eight blocks) keep in shared memory."""
    c = _evict_case(lens, 1, 16, 256, BF, False, 20000, True, seed=7)
    before = {n: None if x is None else x.clone() for n, x in c.items() if n != "page"}
    new_lens, kept = _evict(fa, c, 20000, 1000)
    _settled(fa)
    _check_evict(c, before, new_lens, kept, 20000, 1000)


def test_evict_offsets_past_32_bits(fa):  # noqa: F811
    """A cache of more than 2^31 elements whose last pages are read and written."""
    Hk, d, page, pages = 8, 128, 64, 36000
    k = torch.empty(pages, Hk, page, d, dtype=BF, device="cuda")
    v = torch.empty_like(k)
    w = torch.zeros(pages, Hk, page, device="cuda")
    old, new = [35999, 33000, 5], [35998, 7]
    x = torch.randn(3, Hk, page, d, generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    k[old], v[old] = x, -x
    w[old] = torch.rand(3, Hk, page, generator=torch.Generator().manual_seed(2)).cuda()
    t = lambda l: torch.tensor([l], dtype=torch.int32, device="cuda")
    n, kept = fa.kv_cache_evict(k, v, w, t(old), torch.tensor([180], dtype=torch.int32, device="cuda"), t(new), 100, 10)
    _settled(fa)
    assert n.tolist() == [100]
    for h in range(Hk):
        src = kept[0, h].long()
        flat = x.transpose(0, 1).reshape(Hk, -1, d)[h]
        for cache, sign in ((k, 1), (v, -1)):
            got = cache[new].transpose(0, 1).reshape(Hk, -1, d)[h, :100]
            assert torch.equal(got, sign * flat[src])


def test_evict_streams_and_replayed_graphs(fa):  # noqa: F811
    cs = [_evict_case([300, 20, 150], 2, 64, 16, BF, e, 100, seed=7 + e) for e in (0, 1)]
    befores = [{n: None if x is None else x.clone() for n, x in c.items() if n != "page"} for c in cs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        res = [_evict(fa, c, 100, 9, stream=s) for c, s in zip(cs, streams)]
    _settled(fa)
    for c, before, r in zip(cs, befores, res):
        _check_evict(c, before, *r, 100, 9)
    c, before = cs[0], befores[0]
    new_lens, kept = torch.empty_like(res[0][0]), torch.empty_like(res[0][1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _evict(fa, c, 100, 9, new_lens=new_lens, kept=kept)
    for lens in ([300, 20, 150], [0, 100, 101], [101, 0, 1]):
        for n in ("k", "v", "w"):
            c[n].view(torch.int16 if n != "w" else torch.int32).copy_(before[n].view(torch.int16 if n != "w" else torch.int32))
        c["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        _settled(fa)
        _check_evict(c, before, new_lens, kept, 100, 9)


def test_decode_with_an_evicted_cache(fa):  # noqa: F811
    """As a server runs them: a prompt into the cache, what its last tokens look
    back at, the cache shortened to half, then tokens decoded against it, what they
    attended to added up, and shortened again."""
    from test_gpu_cache import _rows
    for e4m3 in (False, True):
        Hq, Hk, d, page, n, budget, recent, win = 8, 2, 64, 16, 200, 100, 20, 12
        kw = _kw(Hq, 10.0, False)
        k, v = _rows(n + 3, Hk, d, BF, 5, True)
        pages = 40
        mk = lambda: torch.zeros(pages, Hk, page, d, device="cuda").to(torch.float8_e4m3fn if e4m3 else BF)
        sc = lambda: torch.ones(pages, Hk, page, device="cuda") if e4m3 else None
        c = dict(k=mk(), v=mk(), ks=sc(), vs=sc(), page=page)
        t = lambda l: torch.tensor(l, dtype=torch.int32, device="cuda")
        perm = torch.randperm(pages, generator=torch.Generator().manual_seed(2)).tolist()
        c["table"], c["lens"] = t([perm[:13]]), t([n])
        place = lambda table, j: int(table[0, j // page]) * page + j % page
        g = torch.Generator().manual_seed(3)
        fa.kv_cache_write(k[:n], v[:n], torch.tensor([place(c["table"], j) for j in range(n)], device="cuda"), c["k"], c["v"],
                          c["ks"], c["vs"])
        c["q"] = torch.randn(1, win, Hq, d, generator=g).to(BF).cuda() * 3
        def f64():
            for name in ("k", "v"):
                s = c[name + "s"]
                c[name + "_f64"] = _f64(c[name]) * (1.0 if s is None else s.double().cpu().numpy()[..., None])
        f64()
        o, lse = _run(fa, c, 0.125, kw)
        w = _received(fa, c, 0.125, kw, lse, None, torch.full((pages, Hk, page), 7.0, device="cuda"))
        _settled(fa)
        _check(c, 0.125, kw, o, lse)
        _check_received(c, 0.125, kw, lse, None, w)
        for round_, new in enumerate((perm[13:21], perm[21:29])):
            c["w"], c["new"] = w, t([new[:7]])
            before = {x: None if c[x] is None else c[x].clone() for x in ("k", "v", "ks", "vs", "w")}
            new_lens, kept = _evict(fa, c, budget, recent)
            _settled(fa)
            _check_evict(c, before, new_lens, kept, budget, recent)
            c["table"], c["lens"] = t([new]), new_lens
            for step in range(2 if round_ else 1):
                at, row = budget + step, n + round_ + step
                fa.kv_cache_write(k[row:row + 1], v[row:row + 1], torch.tensor([place(c["table"], at)], device="cuda"),
                                  c["k"], c["v"], c["ks"], c["vs"])
                c["lens"] = t([at + 1])
                c["q"] = torch.randn(1, 1, Hq, d, generator=g).to(BF).cuda() * 3
                f64()
                o, lse = _run(fa, c, 0.125, kw)
                past = w.clone()
                _received(fa, c, 0.125, kw, lse, w, w)
                _settled(fa)
                _check(c, 0.125, kw, o, lse)
                r = _ref(c, 0.125, kw, None, lse)
                for j in range(at + 1):
                    p = int(c["table"][0, j // page])
                    old = past[p, :, j % page].double().cpu().numpy() if j < at else 0.0
                    got = w[p, :, j % page].double().cpu().numpy()
                    assert (np.abs(got - old - r["W"][0][:, j]) <= r["tolW"][0][:, j] + 2.0 ** -23 * (np.abs(old) + got) + 1e-37).all()


def test_helpers_refuse_what_does_not_fit(fa):  # noqa: F811
    c = _case(2, 1, 4, 2, 64, 16, [20, 5], BF, True)
    lse = torch.zeros(2, 4, 1, device="cuda")
    w = torch.zeros(c["k"].shape[:3], device="cuda")
    def bad(**kw):
        a = dict(q=c["q"], k_cache=c["k"], block_table=c["table"], seq_lens=c["lens"], lse=lse, scale=0.1, weights=w,
                 k_scale=c["ks"])
        a.update(kw)
        with pytest.raises((ValueError, fa.FlashAttnError)):
            fa.attention_cached_weights(**a)
    bad(q=c["q"].float())
    bad(k_scale=None)
    bad(lse=lse.double())
    bad(lse=lse[:, :2])
    bad(weights=w[:1])
    bad(weights=w.half())
    bad(past=w.cpu())
    bad(past=w[:, :, :8])
    bad(scale=float("nan"))
    bad(softcap=-2.0)
    bad(slopes=torch.zeros(3, device="cuda"))
    bad(seq_lens=c["lens"].long())
    with pytest.raises((ValueError, fa.FlashAttnError)):
        _run(fa, c, 0.1, dict(softcap=2000.0))
    with pytest.raises(ValueError):
        _run(fa, c, 0.1, dict(slopes=torch.zeros(4)))
    e = _evict_case([20, 5], 2, 64, 16, BF, True, 16)
    def bade(budget=16, recent=2, **kw):
        a = dict(k_cache=e["k"], v_cache=e["v"], weights=e["w"], block_table=e["table"], seq_lens=e["lens"],
                 new_table=e["new"], budget=budget, recent=recent, k_scale=e["ks"], v_scale=e["vs"])
        a.update(kw)
        with pytest.raises((ValueError, fa.FlashAttnError)):
            fa.kv_cache_evict(**a)
    bade(budget=0)
    bade(budget=17)
    bade(recent=17)
    bade(recent=-1)
    bade(k_scale=None)
    bade(k_cache=e["k"].float(), v_cache=e["v"].float())
    bade(weights=e["w"].cpu())
    bade(weights=e["w"].double())
    bade(new_table=e["new"].long())
    bade(new_table=e["new"][:1])
    bade(new_lens=torch.zeros(3, dtype=torch.int32, device="cuda"))
    bade(kept=torch.zeros(2, 2, 15, dtype=torch.int32, device="cuda"))
    _settled(fa)
