"""Attention with capped or biased scores, in training and from a paged cache,
and the shortening of such a cache by the attention its tokens got, with the
sizes they are used at.

  prompt   attention over packed sequences whose scores are capped by a tanh, get
           a bias that falls with distance, or see a prefix in both directions
           (attention_packed_fwd with softcap, slopes, prefix_lens)
  train    the same with its gradients (attention_packed_bwd)
  cached   the newest tokens against the paged cache with such scores
           (attention_cached_fwd with softcap, slopes)
  weights  the attention that every cached token got from the newest ones, added
           to what it had before (attention_cached_weights)
  evict    a cache shortened to the tokens with the most of it and the newest
           ones (kv_cache_evict)

Every operator has its plain form here: elementary torch operations in 32 bits
over sequences padded to the longest one, rounded once at the end.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
# cap: the tanh's bound, 0 for none. bias: whether scores fall with distance.
# prefix: whether each sequence has a prefix that all of its tokens see. gain: the
# standard deviation of the scores.

def listed():
    return [
        # the first prompt of an idle server: one short sequence, latency counts
        dict(name="prompt_capped_short", op="prompt", B=1, lo=37, hi=37, empty=0, pad=0, Hq=16, Hk=16, d=64,
             dtype="bf16", causal=True, fused=False, cap=50.0, bias=False, prefix=False, gain=2.0, lens_seed=1),
        # a server's batch of waiting prompts, packed, read out of the fused projection
        dict(name="prompt_capped_mixed", op="prompt", B=24, lo=16, hi=2048, empty=0, pad=0, Hq=32, Hk=8, d=128,
             dtype="bf16", causal=True, fused=True, cap=50.0, bias=False, prefix=False, gain=4.0, lens_seed=2),
        # prompts with a document or an image in front that is seen as a whole, distances biased
        dict(name="prompt_prefix_biased", op="prompt", B=12, lo=64, hi=4096, empty=1, pad=0, Hq=16, Hk=16, d=64,
             dtype="fp16", causal=True, fused=False, cap=0.0, bias=True, prefix=True, gain=1.0, lens_seed=3),
        # fine-tuning on a few short examples, questions seen as a whole
        dict(name="train_biased_short", op="train", B=3, lo=5, hi=200, empty=0, pad=9, Hq=8, Hk=2, d=64,
             dtype="fp16", causal=True, fused=False, cap=0.0, bias=True, prefix=True, gain=1.0, lens_seed=5),
        # a packed training batch of documents of all lengths
        dict(name="train_capped_mixed", op="train", B=16, lo=32, hi=2048, empty=0, pad=0, Hq=32, Hk=8, d=128,
             dtype="bf16", causal=True, fused=True, cap=30.0, bias=False, prefix=False, gain=2.0, lens_seed=6),
        # long-context training
        dict(name="train_capped_long", op="train", B=2, lo=4096, hi=8192, empty=0, pad=0, Hq=32, Hk=8, d=128,
             dtype="bf16", causal=True, fused=False, cap=50.0, bias=False, prefix=False, gain=4.0, lens_seed=7),
        # a serving batch of ragged sequences with an idle place in it
        dict(name="cached_capped_batch", op="cached", B=64, Nq=1, lo=512, hi=8192, empty=1, Hq=32, Hk=8, d=128, page=64,
             dtype="bf16", cache="bf16", cap=50.0, bias=False, gain=4.0, lens_seed=9),
        # long contexts in a quantised cache, distances biased
        dict(name="cached_biased_long", op="cached", B=16, Nq=1, lo=8192, hi=65536, empty=0, Hq=32, Hk=8, d=128,
             page=64, dtype="bf16", cache="e4m3", cap=0.0, bias=True, gain=1.0, lens_seed=10),
        # after a decoding step of a batch: what its tokens attended to is added up
        dict(name="weights_step", op="weights", B=64, Nq=1, lo=512, hi=8192, empty=1, Hq=32, Hk=8, d=128, page=64,
             dtype="bf16", cache="bf16", past=True, cap=50.0, bias=False, gain=4.0, lens_seed=9),
        # after long prompts: what their last tokens look back at
        dict(name="weights_window", op="weights", B=4, Nq=32, lo=4096, hi=16384, empty=0, Hq=32, Hk=8, d=128, page=64,
             dtype="bf16", cache="e4m3", past=False, cap=0.0, bias=False, gain=2.0, lens_seed=11),
        # a batch's caches shortened to a thousand tokens each
        dict(name="evict_batch", op="evict", B=32, lo=512, hi=8192, empty=0, Hk=8, d=128, page=64, dtype="bf16",
             cache="bf16", budget=1024, recent=128, ties=False, lens_seed=12),
        # two long contexts in a quantised cache, to a quarter
        dict(name="evict_long", op="evict", B=2, lo=65536, hi=65536, empty=0, Hk=8, d=128, page=64, dtype="bf16",
             cache="e4m3", budget=16384, recent=1024, ties=True, lens_seed=13),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prompt", "train", "cached", "weights", "evict"])
    Hk = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8])
    Hq = Hk * G if Hk * G <= 32 else Hk * 4
    kind = rng.choice(["cap", "cap", "bias", "both", "prefix"] if op in ("prompt", "train") else ["cap", "bias", "both"])
    score = dict(cap=rng.choice([15.0, 30.0, 50.0]) if kind in ("cap", "both") else 0.0, bias=kind in ("bias", "both"),
                 gain=rng.choice([1.0, 2.0, 4.0, 10.0]))
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op in ("prompt", "train"):
        most, total = (4096, 16384) if op == "prompt" else (2048, 10240)   # longest sequence, tokens in all
        B = _log(rng, 1, 48)
        least = 1 if op == "prompt" else 2               # a lone token's scores have no gradient
        hi = _log(rng, 2 * least, max(2 * least, min(most, total // B)))
        causal = kind == "prefix" or rng.random() < 0.8
        return dict(op=op, B=B, lo=max(least, hi // rng.choice([1, 4, 64])), hi=hi, empty=rng.choice([0, 0, 1]),
                    pad=rng.choice([0, 0, 3, 200]), Hq=Hq, Hk=Hk, d=rng.choice([64, 128, 64, 128, 80, 96, 40]),
                    dtype=dtype, causal=causal, fused=rng.random() < 0.5,
                    prefix=kind == "prefix" or (causal and rng.random() < 0.3), lens_seed=rng.randrange(1 << 30), **score)
    cache = rng.choice(["e4m3", "16"])
    page = rng.choice([16, 32, 64, 128, 256])
    d = rng.choice([64, 128, 64, 128, 80, 96])
    B = _log(rng, 1, 64)
    hi = _log(rng, 8, max(16, 262144 // B // 4))
    at = dict(op=op, B=B, lo=max(1, hi // rng.choice([1, 4, 64])), hi=hi, empty=rng.choice([0, 0, 1]) if B > 1 else 0,
              Hk=Hk, d=d, page=page, dtype=dtype, cache=dtype if cache == "16" else cache,
              lens_seed=rng.randrange(1 << 30))
    if op == "evict":
        budget = _log(rng, 2, hi)
        return dict(at, budget=budget, recent=rng.choice([0, 1, budget // 8, budget // 2]), ties=rng.random() < 0.5)
    if op == "cached":
        return dict(at, Hq=Hq, Nq=rng.choice([1, 1, 1, 2, 4, 7]), **score)
    if rng.random() < 0.3:                               # scores as they are
        score["cap"], score["bias"] = 0.0, False
    return dict(at, Hq=Hq, Nq=rng.choice([1, 1, 4, 16, 33]), past=rng.random() < 0.6, **score)


def _lens(case):
    """Sequence lengths of a case: spread over [lo, hi] by their logarithm,
    `empty` of them zero."""
    rng = random.Random(case["lens_seed"])
    lens = [_log(rng, case["lo"], case["hi"]) for _ in range(case["B"])]
    for _ in range(min(case["empty"], len(lens) - 1)):
        lens[rng.randrange(len(lens))] = 0
    return lens


def _prefixes(case):
    """Prefix lengths of a case's sequences, from none to all of a sequence."""
    rng = random.Random(case["lens_seed"] + 1)
    return [rng.randrange(x + 1) if rng.random() < 0.8 else 0 for x in _lens(case)]


def work(case):
    e = 1 if case.get("cache") == "e4m3" else 2
    d, Hk, lens = case["d"], case["Hk"], _lens(case)
    row = d * e + (4 if e == 1 else 0)                   # a cached row of K or V, with its scale
    if case["op"] == "evict":
        # all weights read; kept rows and their weights read and written, their numbers written
        kept = sum(min(x, case["budget"]) for x in lens)
        return dict(bytes=Hk * (4 * sum(lens) + kept * (4 * row + 4 + 4)), flops=0)
    Hq, n = case["Hq"], sum(lens)
    if case["op"] in ("cached", "weights"):
        B, Nq = case["B"], case["Nq"]
        pairs = sum(sum(max(0, x - i) for i in range(Nq)) for x in lens)
        if case["op"] == "cached":
            return dict(bytes=2 * n * Hk * row + B * Nq * Hq * (4 * d + 4), flops=4 * d * Hq * pairs)
        return dict(bytes=n * Hk * (row + 4 + (4 if case["past"] else 0)) + B * Nq * Hq * (2 * d + 4),
                    flops=2 * d * Hq * pairs)
    if case["causal"]:
        pre = _prefixes(case) if case["prefix"] else [0] * len(lens)
        pairs = sum(x * (x + 1) // 2 + f * (f - 1) // 2 for x, f in zip(lens, pre))
    else:
        pairs = sum(x * x for x in lens)
    rows_q, rows_k = n * Hq * d * 2, n * Hk * d * 2
    if case["op"] == "prompt":
        return dict(bytes=2 * rows_q + 2 * rows_k + 4 * n * Hq, flops=4 * d * Hq * pairs)
    # forward (two products) and backward (five); q, do and k, v in, o, dq and dk, dv and the LSE out
    return dict(bytes=4 * rows_q + 4 * rows_k + 4 * n * Hq, flops=14 * d * Hq * pairs)


# ---------------------------------------------------------------------------
# what a program has in hand
# ---------------------------------------------------------------------------

def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _slopes(Hq, dev):
    """Slopes that fall geometrically over the heads, from 2^(-8 / Hq) to 2^-8."""
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)], dtype=torch.float32, device=dev)


def _heads(g, T, Hq, Hk, d, dtype, fused, gain, dev):
    """q (times gain), k, v of T tokens: tensors of their own, or views of one
    projection."""
    if fused:
        x = torch.randn(T, (Hq + 2 * Hk) * d, generator=g, device=dev)
        x[:, :Hq * d] *= gain
        q, k, v = x.to(dtype).split([Hq * d, Hk * d, Hk * d], dim=1)
        return q.unflatten(1, (Hq, d)), k.unflatten(1, (Hk, d)), v.unflatten(1, (Hk, d))
    return tuple((torch.randn(T, h, d, generator=g, device=dev) * m).to(dtype)
                 for h, m in ((Hq, gain), (Hk, 1.0), (Hk, 1.0)))


def _e4m3_rows(x):
    """Rows of x (float32) as e4m3 with one scale each: the smallest power of
    two that brings the row's largest magnitude to at most 448."""
    m, e = torch.frexp(x.abs().amax(-1))
    scale = torch.ldexp(torch.ones_like(m), e - 9 + (m > 0.875))
    return (x / scale.unsqueeze(-1)).to(torch.float8_e4m3fn), scale


def _paged(g, s, case, lens, more, dev):
    """A paged cache of sequences of these lengths, its pages in no order; `more`
    pages beyond them. Returns the pages left over."""
    page, Hk, d = case["page"], case["Hk"], case["d"]
    need = [-(-x // page) for x in lens]
    pages = sum(need) + more
    perm = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((case["B"], max(1, max(need))), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    for n in ("k", "v") if case["op"] != "weights" else ("k",):
        x = torch.randn(pages, Hk, page, d, generator=g, device=dev)
        if case["cache"] == "e4m3":
            s[n + "_cache"], s[n + "_scale"] = _e4m3_rows(x)
        else:
            s[n + "_cache"], s[n + "_scale"] = x.to(DTYPES[case["cache"]]), None
    s["block_table"] = table
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    return perm[at:]


def prepare(case, seed):
    dev = _device()
    g = torch.Generator(device=dev).manual_seed(seed)
    s = dict(case=case)
    d, Hk, B, lens = case["d"], case["Hk"], case["B"], _lens(case)
    if case["op"] == "evict":
        page = case["page"]
        need = [-(-min(x, case["budget"]) // page) for x in lens]
        spare = _paged(g, s, case, lens, sum(need) + 3, dev)
        new = torch.full((B, -(-case["budget"] // page)), -1, dtype=torch.int32, device=dev)
        at = 0
        for b, n in enumerate(need):
            new[b, :n] = spare[at:at + n]
            at += n
        s["new_table"] = new
        # accumulated attention: a few tokens have most of it, some none
        shape = s["k_cache"].shape[:3]
        w = torch.exp(2.0 * torch.randn(shape, generator=g, device=dev)) * (torch.rand(shape, generator=g, device=dev) > 0.1)
        s["weights"] = w.bfloat16().float() if case["ties"] else w
        s["new_lens"] = torch.zeros(B, dtype=torch.int32, device=dev)
        s["kept"] = torch.full((B, Hk, case["budget"]), -1, dtype=torch.int32, device=dev)
        return s
    Hq = case["Hq"]
    dt = DTYPES[case["dtype"]]
    s["scale"] = d ** -0.5
    s["slopes"] = _slopes(Hq, dev) if case["bias"] else None
    if case["op"] in ("cached", "weights"):
        _paged(g, s, case, lens, 3, dev)
        s["q"] = (torch.randn(B, case["Nq"], Hq, d, generator=g, device=dev) * case["gain"]).to(dt)
        if case["op"] == "weights":
            # the rows' log-sum-exp, as the attention before has left it
            s["v_cache"], s["v_scale"] = s["k_cache"], s["k_scale"]
            s["lse"] = _plain_cached(s)[1]
            shape = s["k_cache"].shape[:3]
            s["past"] = torch.rand(shape, generator=g, device=dev) * 4 if case["past"] else None
            s["weights"] = torch.zeros(shape, device=dev)
        return s
    n = sum(lens)
    T = n + case["pad"]
    s["q"], s["k"], s["v"] = _heads(g, T, Hq, Hk, d, dt, case["fused"], case["gain"], dev)
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    s["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    s["prefix_lens"] = torch.tensor(_prefixes(case), dtype=torch.int32, device=dev) if case["prefix"] else None
    # the longest sequence, and each token's sequence and place in it, for the padded form
    s["longest"] = max(lens)
    s["tok_b"] = torch.repeat_interleave(torch.arange(B), torch.tensor(lens)).to(dev)
    s["tok_i"] = torch.cat([torch.arange(x) for x in lens]).to(dev)
    outs = ["o"]
    if case["op"] == "train":
        s["do"] = torch.randn(T, Hq, d, generator=g, device=dev).to(dt)
        outs += ["dq", "dk", "dv"]
    for name in outs:                                     # rows behind the last sequence stay zero
        s[name] = torch.zeros(T, Hk if name in ("dk", "dv") else Hq, d, dtype=dt, device=dev)
    s["lse"] = torch.zeros(Hq, T, device=dev)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _padded(s, x):
    """[T, h, d] -> float32 [B, h, longest, d], zeros past each sequence."""
    y = torch.zeros(s["case"]["B"], s["longest"], *x.shape[1:], device=x.device)
    y[s["tok_b"], s["tok_i"]] = x[:s["tok_b"].numel()].float()
    return y.transpose(1, 2)


def _packed(s, y, into):
    """float32 [B, h, longest, d] -> the rows of `into`, rounded once; rows
    behind the last sequence are zero."""
    out = torch.zeros_like(into)
    out[:s["tok_b"].numel()] = y.transpose(1, 2)[s["tok_b"], s["tok_i"]].to(into.dtype)
    return out


def _plain_packed(s):
    c = s["case"]
    G, L, dev = c["Hq"] // c["Hk"], s["longest"], s["q"].device
    q = _padded(s, s["q"])
    k, v = (_padded(s, s[n]).repeat_interleave(G, dim=1) for n in ("k", "v"))
    lens = s["cu_seqlens"].diff()
    i = torch.arange(L, device=dev)
    hidden = (i >= lens.view(-1, 1, 1, 1))                # [B, 1, 1, L] over the keys
    if c["causal"]:
        late = i > i.view(-1, 1)
        if c["prefix"]:
            late = late & (i >= s["prefix_lens"].view(-1, 1, 1, 1))
        hidden = hidden | late
    p = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"])
    slope = None                                          # of the cap: 1 - tanh^2
    if c["cap"]:
        p = p.div_(c["cap"]).tanh_()
        if c["op"] == "train":
            slope = 1 - p * p
        p = p.mul_(c["cap"])
    if c["bias"]:
        p = p.sub_(s["slopes"].view(-1, 1, 1) * (i - i.view(-1, 1)).abs().float())
    p = p.masked_fill_(hidden, -math.inf)
    m = p.amax(-1, keepdim=True).clamp_min(-3e38)
    p = p.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    lse = torch.zeros_like(s["lse"])
    lse[:, :s["tok_b"].numel()] = (m + l.log()).squeeze(-1)[s["tok_b"], :, s["tok_i"]].t()
    p = p.div_(l.clamp_min(1e-38))
    o = torch.matmul(p, v)
    out = [_packed(s, o, s["o"]), lse]
    if c["op"] == "train":
        do = _padded(s, s["do"])
        dv = torch.matmul(p.transpose(-1, -2), do).unflatten(1, (c["Hk"], G)).sum(2)
        ds = torch.matmul(do, v.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p)
        if slope is not None:
            ds = ds.mul_(slope)
        dq = torch.matmul(ds, k).mul_(s["scale"])
        dk = torch.matmul(ds.transpose(-1, -2), q).mul_(s["scale"]).unflatten(1, (c["Hk"], G)).sum(2)
        out += [_packed(s, dq, s["dq"]), _packed(s, dk, s["dk"]), _packed(s, dv, s["dv"])]
    return out


def _gathered(s, name):
    """float32 [B, Hk, L, d] rows of a cache, in the order of their tokens."""
    cache, scale, table = s[name + "_cache"], s[name + "_scale"], s["block_table"].long().clamp_min(0)
    if scale is None:
        x = cache[table].float()                          # [B, pages, Hk, page, d]
    else:
        x = cache.view(torch.uint8)[table].view(torch.float8_e4m3fn).float() * scale[table].unsqueeze(-1)
    return x.transpose(1, 2).flatten(2, 3)


def _cached_scores(s, k):
    """[B, Hk, G Nq, L] scores of the newest tokens, -inf where a key is not seen."""
    c = s["case"]
    G, Nq, L, dev = c["Hq"] // c["Hk"], c["Nq"], k.shape[2], k.device
    q = s["q"].float().permute(0, 2, 1, 3).unflatten(1, (c["Hk"], G)).flatten(2, 3)   # [B, Hk, G Nq, d]
    j = torch.arange(L, device=dev)
    at = s["seq_lens"].view(-1, 1) - (Nq - torch.arange(Nq, device=dev))              # [B, Nq] places of the tokens
    at = at.repeat(1, G).view(-1, 1, G * Nq, 1)
    p = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"])
    if c["cap"]:
        p = p.div_(c["cap"]).tanh_().mul_(c["cap"])
    if c["bias"]:
        slopes = s["slopes"].view(1, c["Hk"], G, 1).expand(-1, -1, -1, Nq).reshape(1, c["Hk"], G * Nq, 1)
        p = p.sub_(slopes * (at - j).abs().float())
    return p.masked_fill_(j > at, -math.inf)


def _plain_cached(s):
    c = s["case"]
    G, Nq = c["Hq"] // c["Hk"], c["Nq"]
    p = _cached_scores(s, _gathered(s, "k"))
    m = p.amax(-1, keepdim=True).clamp_min(-3e38)
    p = p.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.div_(l.clamp_min(1e-38)), _gathered(s, "v"))
    o = o.unflatten(2, (G, Nq)).flatten(1, 2).transpose(1, 2).to(s["q"].dtype)        # [B, Nq, Hq, d]
    return [o.contiguous(), (m + l.log()).squeeze(-1).unflatten(2, (G, Nq)).flatten(1, 2).contiguous()]


def _places(s, table, lens):
    """Sequences, token numbers, pages and places of all tokens of a paged cache."""
    page = s["case"]["page"]
    j = torch.arange(table.shape[1] * page, device=table.device)
    b, j = torch.nonzero(j < lens.view(-1, 1), as_tuple=True)
    return b, j, table[b, j.div(page, rounding_mode="floor")].long(), j.remainder(page)


def _plain_weights(s):
    c = s["case"]
    G, Nq = c["Hq"] // c["Hk"], c["Nq"]
    lse = s["lse"].unflatten(1, (c["Hk"], G)).flatten(2, 3).unsqueeze(-1)             # [B, Hk, G Nq, 1]
    w = _cached_scores(s, _gathered(s, "k")).sub_(lse.clamp_min(-3e38)).exp_().sum(2)   # [B, Hk, L]
    b, j, page, at = _places(s, s["block_table"], s["seq_lens"])
    new = w[b, :, j]
    if c["past"]:
        old = (j < s["seq_lens"][b] - Nq).unsqueeze(1)
        new = new + torch.where(old, s["past"][page, :, at], torch.zeros_like(new))
    s["weights"][page, :, at] = new
    return [s["weights"]]


def _plain_evict(s):
    c = s["case"]
    Hk, budget, dev = c["Hk"], c["budget"], s["weights"].device
    n = s["seq_lens"].long().view(-1, 1, 1)
    L = s["block_table"].shape[1] * c["page"]
    w = s["weights"][s["block_table"].long().clamp_min(0)].transpose(1, 2).flatten(2, 3)   # [B, Hk, L]
    j = torch.arange(L, device=dev)
    w = torch.where(j >= n - c["recent"], torch.full_like(w, math.inf), w)            # the newest first
    w = torch.where(j >= n, torch.full_like(w, -1.0), w)
    order = torch.sort(w, dim=2, descending=True, stable=True).indices[:, :, :budget]
    keep = torch.zeros_like(w, dtype=torch.bool).scatter_(2, order, True) & (j < n)
    lens = s["seq_lens"].clamp_max(budget)
    b, h, src = torch.nonzero(keep, as_tuple=True)        # by sequence, head, token
    dst = (keep.cumsum(2) - 1)[b, h, src]
    s["new_lens"].copy_(lens)
    s["kept"].fill_(-1)
    s["kept"][b, h, dst] = src.to(torch.int32)
    p = c["page"]
    from_page, to_page = s["block_table"][b, src // p].long(), s["new_table"][b, dst // p].long()
    out = []
    for name in ("k_cache", "v_cache", "k_scale", "v_scale", "weights"):
        x = s[name]
        if x is not None:
            y = x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x
            y[to_page, h, dst % p] = y[from_page, h, src % p]
            out.append(x)
    return out + [s["new_lens"], s["kept"]]


def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return {"prompt": _plain_packed, "train": _plain_packed, "cached": _plain_cached, "weights": _plain_weights,
                "evict": _plain_evict}[op](s)
    import exact_io_aware_39_gb300 as fa
    if op == "evict":
        fa.kv_cache_evict(s["k_cache"], s["v_cache"], s["weights"], s["block_table"], s["seq_lens"], s["new_table"],
                          c["budget"], c["recent"], k_scale=s["k_scale"], v_scale=s["v_scale"], new_lens=s["new_lens"],
                          kept=s["kept"])
        return [s[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale", "weights", "new_lens", "kept")
                if s[n] is not None]
    if op == "weights":
        fa.attention_cached_weights(s["q"], s["k_cache"], s["block_table"], s["seq_lens"], s["lse"], s["scale"],
                                    s["weights"], k_scale=s["k_scale"], past=s["past"], softcap=c["cap"],
                                    slopes=s["slopes"])
        return [s["weights"]]
    if op == "cached":
        o, lse = fa.attention_cached_fwd(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["seq_lens"],
                                         s["scale"], k_scale=s["k_scale"], v_scale=s["v_scale"], softcap=c["cap"],
                                         slopes=s["slopes"])
        return [o, lse]
    o, lse = fa.attention_packed_fwd(s["q"], s["k"], s["v"], s["cu_seqlens"], s["scale"], causal=c["causal"],
                                     out=s["o"], lse=s["lse"], softcap=c["cap"], slopes=s["slopes"],
                                     prefix_lens=s["prefix_lens"])
    if op == "prompt":
        return [o, lse]
    dq, dk, dv = fa.attention_packed_bwd(s["q"], s["k"], s["v"], o, s["do"], lse, s["cu_seqlens"], s["scale"],
                                         causal=c["causal"], dq=s["dq"], dk=s["dk"], dv=s["dv"], softcap=c["cap"],
                                         slopes=s["slopes"], prefix_lens=s["prefix_lens"])
    return [o, lse, dq, dk, dv]


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _scored(case, s, raw, rows, cols, head):
    """Scores from the products of the queries at `rows` with the keys at `cols`:
    capped, then lowered with the distance."""
    if case["cap"]:
        e = torch.exp(-2.0 * raw.abs() / case["cap"])
        raw = torch.sign(raw) * case["cap"] * (1.0 - e) / (1.0 + e)
    if case["bias"]:
        raw = raw - float(s["slopes"][head]) * torch.abs(rows[:, None] - cols[None, :]).double()
    return raw


def _softmax_rows(scores):
    """Rows of weights and their log-sum-exp; a row without a finite score has
    weights of zero and -inf."""
    top = scores.max(dim=1, keepdim=True).values if scores.shape[1] else scores.new_full((scores.shape[0], 1), -math.inf)
    w = torch.exp(scores - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    total = w.sum(dim=1, keepdim=True)
    return torch.where(total > 0, w / total, torch.zeros_like(w)), (top + torch.log(total)).squeeze(1)


def _exact_packed(case, s):
    c, dev = case, s["q"].device
    T, G = s["q"].shape[0], c["Hq"] // c["Hk"]
    names = ["o"] + (["dq", "dk", "dv"] if c["op"] == "train" else [])
    res = {n: torch.zeros(s[n].shape, dtype=torch.float64, device=dev) for n in names}
    lse = torch.zeros(c["Hq"], T, dtype=torch.float64, device=dev)
    t0 = 0
    for n, first in zip(_lens(c), _prefixes(c)):
        tok = slice(t0, t0 + n)
        t0 += n
        if n == 0:
            continue
        at = torch.arange(n, device=dev)
        visible = torch.ones(n, n, dtype=torch.bool, device=dev)
        if c["causal"]:
            visible = visible.tril()
            if c["prefix"]:
                visible[:, :first] = True
        for h in range(c["Hq"]):
            q, k, v = s["q"][tok, h].double(), s["k"][tok, h // G].double(), s["v"][tok, h // G].double()
            raw = s["scale"] * (q @ k.T)
            w, lse[h, tok] = _softmax_rows(_scored(c, s, raw, at, at, h).masked_fill(~visible, -math.inf))
            o = w @ v
            res["o"][tok, h] = o
            if c["op"] == "train":
                do = s["do"][tok, h].double()
                res["dv"][tok, h // G] += w.T @ do
                ds = w * (do @ v.T - (do * o).sum(dim=1, keepdim=True))
                if c["cap"]:                              # the cap's slope, 1 / cosh^2
                    ds = ds / torch.cosh((raw / c["cap"]).clamp(-300, 300)) ** 2
                res["dq"][tok, h] = s["scale"] * (ds @ k)
                res["dk"][tok, h // G] += s["scale"] * (ds.T @ q)
    return [res["o"], lse] + [res[n] for n in names[1:]]


def _tokens(case, s, name, b, n):
    """Rows [Hk, n, d] of sequence b."""
    used = s["block_table"][b, :-(-n // case["page"])].tolist()
    x = torch.cat([s[name + "_cache"][p].double() for p in used], dim=1)[:, :n]
    if s[name + "_scale"] is not None:
        x = x * torch.cat([s[name + "_scale"][p].double() for p in used], dim=1)[:, :n].unsqueeze(2)
    return x


def _exact_cached(case, s):
    c, dev = case, s["q"].device
    G, Nq = c["Hq"] // c["Hk"], c["Nq"]
    if c["op"] == "cached":
        o = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
        lse = torch.full((c["B"], c["Hq"], Nq), -math.inf, dtype=torch.float64, device=dev)
    else:
        weights = s["weights"].double()
    for b, n in enumerate(_lens(c)):
        if n == 0:
            continue
        k = _tokens(c, s, "k", b, n)
        v = _tokens(c, s, "v", b, n) if c["op"] == "cached" else None
        cols = torch.arange(n, device=dev)
        got = torch.zeros(c["Hk"], n, dtype=torch.float64, device=dev)
        rows = torch.arange(n - Nq, n, device=dev)        # places of the newest tokens
        for h in range(c["Hq"]):
            score = _scored(c, s, s["scale"] * (s["q"][b, :, h].double() @ k[h // G].T), rows, cols, h)
            score = score.masked_fill(cols[None, :] > rows[:, None], -math.inf)
            if c["op"] == "cached":
                w, lse[b, h] = _softmax_rows(score)
                o[b, :, h] = w @ v[h // G]
            else:
                live = rows >= 0                          # (a token before the first sees nothing)
                got[h // G] += torch.exp(score[live] - s["lse"][b, h, live].double()[:, None]).sum(dim=0)
        if c["op"] == "weights":
            for j0 in range(0, n, c["page"]):
                j1 = min(n, j0 + c["page"])
                page = int(s["block_table"][b, j0 // c["page"]])
                w = got[:, j0:j1]
                if c["past"]:
                    w = w + torch.where(cols[j0:j1] < n - Nq, s["past"][page, :, :j1 - j0].double(), 0.0)
                weights[page, :, :j1 - j0] = w
    return [o, lse] if c["op"] == "cached" else [weights]


def _exact_evict(case, s):
    c = case
    page, budget = c["page"], c["budget"]
    names = [n for n in ("k_cache", "v_cache", "k_scale", "v_scale", "weights") if s[n] is not None]
    out = {n: s[n].double() for n in names}
    new_lens = torch.zeros_like(s["new_lens"])
    kept = torch.full_like(s["kept"], -1)
    old_table, new_table, w = s["block_table"].tolist(), s["new_table"].tolist(), s["weights"].tolist()
    for b, n in enumerate(_lens(c)):
        new_lens[b] = min(n, budget)
        for h in range(c["Hk"]):
            tokens = list(range(n))
            if n > budget:
                older = n - c["recent"]
                by_weight = sorted(range(older), key=lambda j: (-w[old_table[b][j // page]][h][j % page], j))
                tokens = sorted(by_weight[:budget - c["recent"]]) + tokens[older:]
            kept[b, h, :len(tokens)] = torch.tensor(tokens, dtype=torch.int32)
            src = torch.tensor([old_table[b][j // page] * page + j % page for j in tokens], dtype=torch.long)
            dst = torch.tensor([new_table[b][i // page] * page + i % page for i in range(len(tokens))], dtype=torch.long)
            src, dst = src.to(s["weights"].device), dst.to(s["weights"].device)
            for n_ in names:
                out[n_][dst // page, h, dst % page] = s[n_][src // page, h, src % page].double()
    return [out[n] for n in names] + [new_lens, kept]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    return _exact_evict(case, s) if op == "evict" else _exact_cached(case, s) if op in ("cached", "weights") else _exact_packed(case, s)
