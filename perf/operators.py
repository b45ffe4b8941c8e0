"""Attention operators of training on packed batches and of serving from a
paged key/value cache, with the sizes they are used at.

  prompt  attention over packed sequences of different lengths, causal or not,
          with grouped key/value heads (attention_packed_fwd)
  train   the same with its gradients (attention_packed_fwd, attention_packed_bwd)
  write   keys and values written into a paged cache, as 16-bit values or
          quantised to e4m3 with one scale per token and head (kv_cache_write)
  cached  the newest token, or the newest few, of every sequence against the
          paged cache (attention_cached_fwd)

Every operator has its plain form here: elementary torch operations in 32 bits
over sequences padded to the longest one, rounded once at the end.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
E4M3_MAX = 448.0
E4M3_MIN_EXP = -64      # the smallest scale is 2^-64


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the first prompt of an idle server: one short sequence, latency counts
        dict(name="prompt_one_short", op="prompt", B=1, lo=37, hi=37, empty=0, pad=0, Hq=16, Hk=16, d=64,
             dtype="bf16", causal=True, fused=False, lens_seed=1),
        # a server's batch of waiting prompts, packed, read out of the fused projection
        dict(name="prompt_mixed", op="prompt", B=24, lo=16, hi=2048, empty=0, pad=0, Hq=32, Hk=8, d=128,
             dtype="bf16", causal=True, fused=True, lens_seed=2),
        # one long document
        dict(name="prompt_long", op="prompt", B=1, lo=16384, hi=16384, empty=0, pad=0, Hq=32, Hk=8, d=128,
             dtype="bf16", causal=True, fused=False, lens_seed=3),
        # an encoder's batch without padding, both directions visible
        dict(name="encoder_packed", op="prompt", B=32, lo=128, hi=512, empty=0, pad=0, Hq=16, Hk=16, d=64,
             dtype="fp16", causal=False, fused=False, lens_seed=4),
        # fine-tuning on a few short examples
        dict(name="train_short", op="train", B=3, lo=5, hi=200, empty=0, pad=9, Hq=8, Hk=2, d=64,
             dtype="fp16", causal=True, fused=False, lens_seed=5),
        # a packed training batch of documents of all lengths
        dict(name="train_mixed", op="train", B=16, lo=32, hi=2048, empty=0, pad=0, Hq=32, Hk=8, d=128,
             dtype="bf16", causal=True, fused=True, lens_seed=6),
        # long-context training
        dict(name="train_long", op="train", B=2, lo=4096, hi=8192, empty=0, pad=0, Hq=32, Hk=8, d=128,
             dtype="bf16", causal=True, fused=False, lens_seed=7),
        # one decoding step of a batch: a token per sequence goes into the cache
        dict(name="write_step", op="write", T=64, Hk=8, d=128, page=16, pages=2048, skip=0, dtype="bf16",
             cache="e4m3", fused=True),
        # the prompts of a batch go into the cache
        dict(name="write_prompts", op="write", T=32768, Hk=8, d=128, page=64, pages=600, skip=100, dtype="bf16",
             cache="e4m3", fused=True),
        # one user's chat: a single sequence, latency counts
        dict(name="cached_one", op="cached", B=1, Nq=1, lo=500, hi=500, empty=0, Hq=32, Hk=8, d=128, page=16,
             dtype="bf16", cache="bf16", lens_seed=8),
        # a serving batch of ragged sequences with an idle place in it
        dict(name="cached_batch", op="cached", B=64, Nq=1, lo=512, hi=8192, empty=1, Hq=32, Hk=8, d=128, page=64,
             dtype="bf16", cache="bf16", lens_seed=9),
        # long contexts in a quantised cache
        dict(name="cached_long_e4m3", op="cached", B=16, Nq=1, lo=8192, hi=65536, empty=0, Hq=32, Hk=8, d=128,
             page=64, dtype="bf16", cache="e4m3", lens_seed=10),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prompt", "train", "write", "cached"])
    Hk = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8])
    Hq = Hk * G if Hk * G <= 40 else Hk * 4
    if op in ("prompt", "train"):
        most = 8192 if op == "prompt" else 4096          # longest sequence
        B = _log(rng, 1, 48)
        least = 1 if op == "prompt" else 2               # a lone token's scores have no gradient
        hi = _log(rng, 2 * least, max(2 * least, min(most, 24576 // B)))
        return dict(op=op, B=B, lo=max(least, hi // rng.choice([1, 4, 64])), hi=hi, empty=rng.choice([0, 0, 1]),
                    pad=rng.choice([0, 0, 3, 200]), Hq=Hq, Hk=Hk, d=rng.choice([64, 128, 64, 128, 80, 96, 40]),
                    dtype=rng.choice(["bf16", "bf16", "fp16"]), causal=rng.random() < 0.75,
                    fused=rng.random() < 0.5, lens_seed=rng.randrange(1 << 30))
    cache = rng.choice(["e4m3", "16"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    page = rng.choice([16, 32, 64, 128, 256])
    d = rng.choice([64, 128, 64, 128, 80, 96])
    if op == "write":
        T = _log(rng, 1, 32768)
        return dict(op=op, T=T, Hk=Hk, d=d, page=page, pages=-(-T // page) + rng.randrange(4, 200),
                    skip=rng.choice([0, 0, T // 8]), dtype=dtype, cache=dtype if cache == "16" else cache,
                    fused=rng.random() < 0.5)
    B = _log(rng, 1, 64)
    hi = _log(rng, 8, max(16, 262144 // B // 4))
    return dict(op=op, B=B, Nq=rng.choice([1, 1, 1, 2, 4, 7]), lo=max(1, hi // rng.choice([1, 4, 64])), hi=hi,
                empty=rng.choice([0, 0, 1]) if B > 1 else 0, Hq=Hq, Hk=Hk, d=d, page=page, dtype=dtype,
                cache=dtype if cache == "16" else cache, lens_seed=rng.randrange(1 << 30))


def _lens(case):
    """Sequence lengths of a case: spread over [lo, hi] by their logarithm,
    `empty` of them zero."""
    rng = random.Random(case["lens_seed"])
    lens = [_log(rng, case["lo"], case["hi"]) for _ in range(case["B"])]
    for i in range(min(case["empty"], len(lens) - 1)):
        lens[rng.randrange(len(lens))] = 0
    return lens


def work(case):
    e = 1 if case.get("cache") == "e4m3" else 2
    d, Hk = case["d"], case["Hk"]
    if case["op"] == "write":
        # keys and values read once and written once, one 4-byte scale per row in e4m3
        return dict(bytes=2 * case["T"] * Hk * (d * (2 + e) + (4 if e == 1 else 0)) + 8 * case["T"], flops=0)
    lens, Hq = _lens(case), case["Hq"]
    if case["op"] == "cached":
        n, B, Nq = sum(lens), case["B"], case["Nq"]
        pairs = sum(sum(max(0, x - i) for i in range(Nq)) for x in lens)
        return dict(bytes=2 * n * Hk * (d * e + (4 if e == 1 else 0)) + B * Nq * Hq * (4 * d + 4),
                    flops=4 * d * Hq * pairs)
    n = sum(lens)
    pairs = sum(x * (x + 1) // 2 if case["causal"] else x * x for x in lens)
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


def _heads(g, T, Hq, Hk, d, dtype, fused, dev):
    """q, k, v of T tokens: tensors of their own, or views of one projection."""
    if fused:
        x = torch.randn(T, (Hq + 2 * Hk) * d, generator=g, device=dev).to(dtype)
        q, k, v = x.split([Hq * d, Hk * d, Hk * d], dim=1)
        return q.unflatten(1, (Hq, d)), k.unflatten(1, (Hk, d)), v.unflatten(1, (Hk, d))
    return tuple(torch.randn(T, h, d, generator=g, device=dev).to(dtype) for h in (Hq, Hk, Hk))


def _e4m3_rows(x):
    """Rows of x (float32) as e4m3 with one scale each: the smallest power of
    two that brings the row's largest magnitude to at most 448 (2^-64 at least)."""
    m, e = torch.frexp(x.abs().amax(-1))
    e = e - 9 + (m > 0.875)
    e = torch.where(m > 0, e, torch.full_like(e, E4M3_MIN_EXP)).clamp_min(E4M3_MIN_EXP)
    scale = torch.ldexp(torch.ones_like(m), e)
    return (x / scale.unsqueeze(-1)).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    dev = _device()
    g = torch.Generator(device=dev).manual_seed(seed)
    s = dict(case=case)
    d, Hk = case["d"], case["Hk"]
    if case["op"] == "write":
        T, page, pages = case["T"], case["page"], case["pages"]
        dt = DTYPES[case["dtype"]]
        _, s["k"], s["v"] = _heads(g, T, Hk, Hk, d, dt, case["fused"], dev)
        slots = torch.randperm(pages * page, generator=g, device=dev)[:T]
        if case["skip"]:                                  # padding tokens, not written
            slots[torch.randperm(T, generator=g, device=dev)[:case["skip"]]] = -1
        s["slots"] = slots
        ct = DTYPES[case["cache"]]
        for n in ("k_cache", "v_cache"):
            s[n] = torch.randn(pages, Hk, page, d, generator=g, device=dev).to(ct)
        for n in ("k_scale", "v_scale"):
            s[n] = torch.ones(pages, Hk, page, device=dev) if case["cache"] == "e4m3" else None
        return s
    lens, B, Hq = _lens(case), case["B"], case["Hq"]
    dt = DTYPES[case["dtype"]]
    s["scale"] = d ** -0.5
    if case["op"] == "cached":
        page, Nq = case["page"], case["Nq"]
        need = [-(-x // page) for x in lens]
        width, pages = max(1, max(need)), sum(need) + 3
        perm = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
        table = torch.full((B, width), -1, dtype=torch.int32, device=dev)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = perm[at:at + n]
            at += n
        s["q"] = torch.randn(B, Nq, Hq, d, generator=g, device=dev).to(dt)
        for n in ("k", "v"):
            x = torch.randn(pages, Hk, page, d, generator=g, device=dev)
            if case["cache"] == "e4m3":
                s[n + "_cache"], s[n + "_scale"] = _e4m3_rows(x)
            else:
                s[n + "_cache"], s[n + "_scale"] = x.to(dt), None
        s["block_table"] = table
        s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        return s
    n = sum(lens)
    T = n + case["pad"]
    s["q"], s["k"], s["v"] = _heads(g, T, Hq, Hk, d, dt, case["fused"], dev)
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    s["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device=dev)
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
        hidden = hidden | (i > i.view(-1, 1))
    p = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"]).masked_fill_(hidden, -math.inf)
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
        dq = torch.matmul(ds, k).mul_(s["scale"])
        dk = torch.matmul(ds.transpose(-1, -2), q).mul_(s["scale"]).unflatten(1, (c["Hk"], G)).sum(2)
        out += [_packed(s, dq, s["dq"]), _packed(s, dk, s["dk"]), _packed(s, dv, s["dv"])]
    return out


def _plain_write(s):
    c = s["case"]
    keep = s["slots"] >= 0
    slots = s["slots"][keep]
    page, at = slots.div(c["page"], rounding_mode="floor"), slots.remainder(c["page"])
    out = []
    for n in ("k", "v"):
        rows, cache, scale = s[n][keep], s[n + "_cache"], s[n + "_scale"]
        out.append(cache)
        if scale is not None:
            rows, sc = _e4m3_rows(rows.float())
            scale[page, :, at] = sc
            rows, cache = rows.view(torch.uint8), cache.view(torch.uint8)
            out.append(scale)
        cache[page, :, at] = rows
    return out


def _plain_cached(s):
    c = s["case"]
    G, Nq, page = c["Hq"] // c["Hk"], c["Nq"], c["page"]
    table = s["block_table"].long().clamp_min(0)
    L, dev = table.shape[1] * page, table.device
    kv = []
    for n in ("k", "v"):
        x = s[n + "_cache"][table] if s[n + "_scale"] is None else s[n + "_cache"].view(torch.uint8)[table].view(
            torch.float8_e4m3fn)
        x = x.float()                                     # [B, pages, Hk, page, d]
        if s[n + "_scale"] is not None:
            x = x * s[n + "_scale"][table].unsqueeze(-1)
        kv.append(x.transpose(1, 2).flatten(2, 3))        # [B, Hk, L, d]
    q = s["q"].float().permute(0, 2, 1, 3).unflatten(1, (c["Hk"], G)).flatten(2, 3)   # [B, Hk, G Nq, d]
    j = torch.arange(L, device=dev)
    seen = s["seq_lens"].view(-1, 1) - (Nq - 1 - torch.arange(Nq, device=dev))        # [B, Nq] keys of each token
    hidden = j >= seen.repeat(1, G).view(-1, 1, G * Nq, 1)
    p = torch.matmul(q, kv[0].transpose(-1, -2)).mul_(s["scale"]).masked_fill_(hidden, -math.inf)
    m = p.amax(-1, keepdim=True).clamp_min(-3e38)
    p = p.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.div_(l.clamp_min(1e-38)), kv[1])
    o = o.unflatten(2, (G, Nq)).flatten(1, 2).transpose(1, 2).to(s["q"].dtype)        # [B, Nq, Hq, d]
    return [o.contiguous(), (m + l.log()).squeeze(-1).unflatten(2, (G, Nq)).flatten(1, 2)]


def run(s):
    op = s["case"]["op"]
    if not own:
        return _plain_write(s) if op == "write" else _plain_cached(s) if op == "cached" else _plain_packed(s)
    import exact_io_aware_39_gb300 as fa
    if op == "write":
        fa.kv_cache_write(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], k_scale=s["k_scale"],
                          v_scale=s["v_scale"])
        return [s[n] for n in ("k_cache", "k_scale", "v_cache", "v_scale") if s[n] is not None]
    if op == "cached":
        o, lse = fa.attention_cached_fwd(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["seq_lens"],
                                         s["scale"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        return [o, lse]
    o, lse = fa.attention_packed_fwd(s["q"], s["k"], s["v"], s["cu_seqlens"], s["scale"], causal=s["case"]["causal"],
                                     out=s["o"], lse=s["lse"])
    if op == "prompt":
        return [o, lse]
    dq, dk, dv = fa.attention_packed_bwd(s["q"], s["k"], s["v"], o, s["do"], lse, s["cu_seqlens"], s["scale"],
                                         causal=s["case"]["causal"], dq=s["dq"], dk=s["dk"], dv=s["dv"])
    return [o, lse, dq, dk, dv]


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _softmax_rows(scores):
    """Rows of weights and their log-sum-exp; a row without a finite score has
    weights of zero and -inf."""
    top = scores.max(dim=1, keepdim=True).values if scores.shape[1] else scores.new_full((scores.shape[0], 1), -math.inf)
    w = torch.exp(scores - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    total = w.sum(dim=1, keepdim=True)
    return torch.where(total > 0, w / total, torch.zeros_like(w)), (top + torch.log(total)).squeeze(1)


def _exact_packed(case, s):
    c = case
    T, G = s["q"].shape[0], c["Hq"] // c["Hk"]
    names = ["o"] + (["dq", "dk", "dv"] if c["op"] == "train" else [])
    res = {n: torch.zeros(s[n].shape, dtype=torch.float64, device=s["q"].device) for n in names}
    lse = torch.zeros(c["Hq"], T, dtype=torch.float64, device=s["q"].device)
    t0 = 0
    for n in _lens(c):
        rows = slice(t0, t0 + n)
        t0 += n
        if n == 0:
            continue
        visible = torch.ones(n, n, dtype=torch.bool, device=s["q"].device)
        if c["causal"]:
            visible = visible.tril()
        for h in range(c["Hq"]):
            q, k, v = s["q"][rows, h].double(), s["k"][rows, h // G].double(), s["v"][rows, h // G].double()
            scores = (s["scale"] * (q @ k.T)).masked_fill(~visible, -math.inf)
            w, lse[h, rows] = _softmax_rows(scores)
            o = w @ v
            res["o"][rows, h] = o
            if c["op"] == "train":
                do = s["do"][rows, h].double()
                res["dv"][rows, h // G] += w.T @ do
                ds = w * (do @ v.T - (do * o).sum(dim=1, keepdim=True))
                res["dq"][rows, h] = s["scale"] * (ds @ k)
                res["dk"][rows, h // G] += s["scale"] * (ds.T @ q)
    return [res["o"], lse] + [res[n] for n in names[1:]]


def _exact_write(case, s):
    c, out = case, []
    slots = s["slots"].tolist()
    t = torch.tensor([i for i, x in enumerate(slots) if x >= 0], dtype=torch.long, device=s["k"].device)
    at = s["slots"][t]
    for n in ("k", "v"):
        rows, cache = s[n][t].double(), s[n + "_cache"].double()
        flat = cache.permute(0, 2, 1, 3).reshape(-1, c["Hk"], c["d"])
        scales = None
        if c["cache"] == "e4m3":
            # the smallest power of two with |row| <= 448 scale, from its logarithm
            top = rows.abs().amax(dim=2)
            e = torch.ceil(torch.log2(top.clamp_min(1e-300) / E4M3_MAX))
            e = torch.where(top > E4M3_MAX * torch.exp2(e), e + 1, e)
            e = torch.where(top <= E4M3_MAX * torch.exp2(e - 1), e - 1, e).clamp_min(E4M3_MIN_EXP)
            scales = s[n + "_scale"].double().permute(0, 2, 1).reshape(-1, c["Hk"])
            scales[at] = torch.exp2(e)
            y = rows / torch.exp2(e).unsqueeze(2)
            # e4m3: three bits behind the leading one, steps of 2^-9 below 2^-6
            step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
            rows = torch.round(y / step) * step
            scales = scales.reshape(c["pages"], c["page"], c["Hk"]).permute(0, 2, 1).contiguous()
        flat[at] = rows
        out.append(flat.reshape(c["pages"], c["page"], c["Hk"], c["d"]).permute(0, 2, 1, 3).contiguous())
        if scales is not None:
            out.append(scales)
    return out


def _exact_cached(case, s):
    c = case
    G, Nq = c["Hq"] // c["Hk"], c["Nq"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.full((c["B"], c["Hq"], Nq), -math.inf, dtype=torch.float64, device=s["q"].device)
    for b, n in enumerate(_lens(c)):
        used = s["block_table"][b, :-(-n // c["page"])].tolist()
        if not used:
            continue
        kv = []
        for name in ("k", "v"):
            x = torch.cat([s[name + "_cache"][p].double() for p in used], dim=1)[:, :n]
            if s[name + "_scale"] is not None:
                x = x * torch.cat([s[name + "_scale"][p].double() for p in used], dim=1)[:, :n].unsqueeze(2)
            kv.append(x)
        for i in range(Nq):
            m = max(0, n - (Nq - 1 - i))
            for h in range(c["Hk"]):
                q = s["q"][b, i, h * G:(h + 1) * G].double()
                w, lse[b, h * G:(h + 1) * G, i] = _softmax_rows(s["scale"] * (q @ kv[0][h, :m].T))
                o[b, i, h * G:(h + 1) * G] = w @ kv[1][h, :m]
    return [o, lse]


def exact(case, seed):
    s = prepare(case, seed)
    return {"write": _exact_write, "cached": _exact_cached}.get(case["op"], _exact_packed)(case, s)
