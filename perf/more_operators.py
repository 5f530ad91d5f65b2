"""Attention with sinks and over shared prefixes, as cases that can be timed and checked.

A sliding window forgets a sequence's first tokens, although a trained model keeps sending them a
large part of its attention.  With `sinks` = S the first S tokens of a sequence stay visible to every
query behind them, in training and in serving; and a batch whose sequences begin with the same long
text (a system prompt, a document that many questions are asked about) holds that text's pages once:

  fwd      training forward: each query sees the window's keys and the sinks; o and the log-sum-exp
  bwd      its gradients dq, dk, dv (a sink's dk and dv are sums over every query behind it)
  token    serving: one token, or a few that are verified at once, over the paged 8-bit cache, seeing
           the window's slots and the sinks; optionally adding the weights that cached tokens received
  shared   serving: the same for a batch whose tables begin with the same `shared` pages, which are
           walked once for all sequences

`run` computes each in plain torch operations in 32 bits, or, with `own`, by the library's calls.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # The long sliding-window layer with four sinks, as such models are trained.
        dict(name="fwd long", op="fwd", B=1, Hq=32, Hkv=16, Lq=32768, Lk=32768, D=128, window=1024,
             sinks=4, causal=True, dtype="bf16"),
        # Wide heads, a block of learned first tokens as sinks, a length that no tile divides.
        dict(name="fwd d256", op="fwd", B=1, Hq=32, Hkv=16, Lq=8191, Lk=8191, D=256, window=1024,
             sinks=129, causal=True, dtype="fp16"),
        # A short suffix of a short prompt, narrow heads: latency.
        dict(name="fwd suffix", op="fwd", B=2, Hq=4, Hkv=2, Lq=255, Lk=1000, D=64, window=64,
             sinks=1, causal=True, dtype="fp16"),
        # The longest example's step of the long layer.
        dict(name="bwd long", op="bwd", B=1, Hq=32, Hkv=16, Lq=30553, Lk=30553, D=128, window=1024,
             sinks=4, causal=True, dtype="bf16"),
        # Wide heads.
        dict(name="bwd d256", op="bwd", B=1, Hq=32, Hkv=16, Lq=8191, Lk=8191, D=256, window=1024,
             sinks=129, causal=True, dtype="fp16"),
        # A few short sequences, an odd number of query heads to a kv head, narrow heads.
        dict(name="bwd short", op="bwd", B=4, Hq=12, Hkv=4, Lq=512, Lk=512, D=64, window=128,
             sinks=16, causal=True, dtype="bf16"),
        # One user, one token, a sliding layer: the smallest call of a decode loop.
        dict(name="token", op="token", B=1, Hq=32, Hkv=16, D=128, page=64, T=1, shortest=32768,
             longest=32768, window=1024, sinks=4, ragged=False, acc=False, dtype="bf16", spread=1),
        # A batch server's sliding layer, contexts from short to long, a few drafted tokens of each
        # sequence, weights accumulated.
        dict(name="token batch", op="token", B=64, Hq=32, Hkv=8, D=128, page=64, T=4, shortest=3,
             longest=30553, window=4096, sinks=68, ragged=True, acc=True, dtype="bf16", spread=2),
        # Wide heads, a middling batch, one token each.
        dict(name="token d256", op="token", B=12, Hq=32, Hkv=16, D=256, page=32, T=1, shortest=700,
             longest=30553, window=1024, sinks=4, ragged=False, acc=False, dtype="fp16", spread=3),
        # Many short conversations that follow one long document, in a full layer.
        dict(name="shared batch", op="shared", B=64, Hq=32, Hkv=8, D=128, page=64, T=1,
             prefix=32768, shortest=1, longest=1024, window=0, sinks=0, ragged=False, dtype="bf16",
             spread=4),
        # A system prompt before longer conversations, drafted tokens, wide heads, a sliding layer
        # whose window still reaches into the prompt for some of them.
        dict(name="shared verify d256", op="shared", B=12, Hq=32, Hkv=16, D=256, page=32, T=5,
             prefix=4096, shortest=5, longest=3000, window=4096, sinks=4, ragged=True,
             dtype="fp16", spread=5),
        # A handful of answers sampled from one short prompt.
        dict(name="shared few", op="shared", B=4, Hq=8, Hkv=2, D=64, page=64, T=1, prefix=960,
             shortest=1, longest=100, window=0, sinks=0, ragged=False, dtype="bf16", spread=6),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["fwd", "bwd", "token", "shared", "shared"])
    D = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    dtype = rng.choice(["bf16", "fp16"])
    if op in ("fwd", "bwd"):
        Hkv = min(Hkv, 8)
        G = rng.choice([1, 2, 3, 4, 8])
        B = rng.choice([1, 1, 2, 3])
        Lk = _log_int(rng, 2, min(16384, (3 << 24) // (B * G * Hkv * D)))
        Lq = Lk if rng.random() < 0.6 else _log_int(rng, 1, Lk)
        causal = rng.random() < 0.8
        return dict(op=op, B=B, Hq=G * Hkv, Hkv=Hkv, Lq=Lq, Lk=Lk, D=D,
                    window=_log_int(rng, 1, min(Lk, 2048 if causal else 1024)),
                    sinks=_log_int(rng, 1, 300), causal=causal, dtype=dtype)
    page = rng.choice([32, 64, 64, 128])
    T = rng.choice([1, 1, 1, 2, 3, 5, 8])
    G = rng.choice([1, 2, 4, 7, 8])
    spread = rng.randrange(1000)
    if op == "token":
        longest = _log_int(rng, 16, 65536)
        B = _log_int(rng, 1, max(1, min(96, (1 << 30) // (longest * Hkv * D))))
        return dict(op=op, B=B, Hq=G * Hkv, Hkv=Hkv, D=D, page=page, T=T,
                    shortest=_log_int(rng, 1, longest), longest=longest,
                    window=_log_int(rng, 1, 4096), sinks=_log_int(rng, 1, 300),
                    ragged=T > 1 and rng.random() < 0.5, acc=rng.random() < 0.5, dtype=dtype,
                    spread=spread)
    prefix = page * max(1, _log_int(rng, 64, 32768) // page)
    longest = _log_int(rng, 16, 4096)
    B = _log_int(rng, 1, max(1, min(96, (1 << 31) // (prefix * Hkv * D),
                                    (1 << 30) // (longest * Hkv * D),
                                    (1 << 30) // (prefix * G * Hkv * T))))
    window = rng.choice([0, 0, _log_int(rng, 16, 2 * prefix)])
    return dict(op=op, B=B, Hq=G * Hkv, Hkv=Hkv, D=D, page=page, T=T, prefix=prefix,
                shortest=_log_int(rng, 1, longest), longest=longest, window=window,
                sinks=_log_int(rng, 1, 300) if window and rng.random() < 0.5 else 0,
                ragged=T > 1 and rng.random() < 0.5, dtype=dtype, spread=spread)


# ---- sizes that follow from a case alone -------------------------------------------------------

def _lengths(c):
    """(tokens in the cache before the call, new tokens) of each sequence; with a shared prefix,
    behind that prefix."""
    r = random.Random(c["spread"])
    lens = [max(0, r.randint(c["shortest"], c["longest"]) - c["T"]) for _ in range(c["B"])]
    new = [r.randint(0, c["T"]) if c["ragged"] else c["T"] for _ in range(c["B"])]
    return [n + c.get("prefix", 0) for n in lens], new


def _seen(at, window, sinks):
    """Slots that a query at slot `at` sees: (window's first slot, sinks before it)."""
    lo = max(0, at - window + 1)
    return lo, min(sinks, lo)


def _pairs(c):
    """Visible (query, key) pairs of one head."""
    n, off, W = 0, c["Lk"] - c["Lq"], c["window"]
    for p in range(off, c["Lk"]):
        lo, s = _seen(p, W, c["sinks"])
        n += s + (p if c["causal"] else min(c["Lk"] - 1, p + W - 1)) - lo + 1
    return n


def work(case):
    c = case
    D = c["D"]
    if c["op"] in ("fwd", "bwd"):
        rows, keys = c["B"] * c["Hq"] * c["Lq"], c["B"] * c["Hkv"] * c["Lk"]
        n = _pairs(c) * c["B"] * c["Hq"]
        if c["op"] == "fwd":
            return {"bytes": rows * (4 * D + 4) + keys * 4 * D, "flops": 4 * D * n}
        return {"bytes": rows * (8 * D + 4) + keys * 8 * D, "flops": 10 * D * n}
    lens, new = _lengths(c)
    W, P = c["window"] or 1 << 30, c.get("prefix", 0)
    keys = pairs = 0
    first, sunk = P, 0  # of the prefix: the earliest slot that some window sees, and the sinks
    for a, m in zip(lens, new):
        if not m:
            continue
        lo, s = _seen(a, W, c["sinks"])
        most = min(c["sinks"], _seen(a + m - 1, W, c["sinks"])[0])
        keys += a + m - max(lo, P) + max(0, min(most, lo) - P)
        first, sunk = min(first, lo), max(sunk, min(most, P))
        for t in range(m):
            lo, s = _seen(a + t, W, c["sinks"])
            pairs += a + t + 1 - lo + s
    if P:
        keys += P - first + min(sunk, first)
    rows = c["B"] * c["Hq"] * c["T"]
    return {"bytes": keys * c["Hkv"] * (2 * D + 8 * c.get("acc", False) + 8 / c["page"]) +
            rows * (4 * D + 4), "flops": 4 * D * pairs * c["Hq"]}


# ---- inputs ------------------------------------------------------------------------------------

def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[c["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    s = {"case": c}
    B, Hq, Hkv, D = c["B"], c["Hq"], c["Hkv"], c["D"]
    if c["op"] in ("fwd", "bwd"):
        s["q"] = normal(B, Hq, c["Lq"], D).to(dt)
        k = normal(B, Hkv, c["Lk"], D)
        # Trained sinks have keys of their own length and draw weight from every query.
        k[:, :, :c["sinks"]] *= 1.5
        s["k"] = k.to(dt)
        s["v"] = normal(B, Hkv, c["Lk"], D).to(dt)
        if c["op"] == "bwd":
            s["do"] = (normal(B, Hq, c["Lq"], D) * 0.1).to(dt)
            s["o"], s["lse"] = _forward(s["q"], s["k"], s["v"], c)  # the state that training keeps
        return s
    lens, new = _lengths(c)
    page, T, P = c["page"], c["T"], c.get("prefix", 0)
    n, common = -(-(max(lens) + T) // page), P // page
    total = B * (n - common) + common + 1  # the last page belongs to nobody
    # Codes as quantised activations have them: nearly normal, the largest of a block near 448.
    for name in ("k", "v"):
        s[name] = (normal(total, Hkv, page, D) * 100).clamp_(-448, 448).to(torch.float8_e4m3fn)
        s[name + "_scale"] = torch.exp2(torch.randint(-8, -5, (total, Hkv), generator=g,
                                                      device="cuda").float())
    s["weight"] = torch.exp(2 * normal(total, Hkv, page)) if c.get("acc") else None
    order = torch.randperm(total - 1, generator=g, device="cuda").to(torch.int32)
    s["table"] = torch.cat([order[:common].expand(B, common), order[common:].view(B, n - common)],
                           1).contiguous()
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["new"] = torch.tensor(new, dtype=torch.int32, device="cuda") if c["ragged"] else None
    s["q"] = normal(B, Hq, T, D).to(dt)
    return s


# ---- one pass ----------------------------------------------------------------------------------

def run(state):
    s, c = state, state["case"]
    if own:
        import sliding_window_flash_gb300 as swa
        if c["op"] == "fwd":
            return list(swa.swa_attn_fwd(s["q"], s["k"], s["v"], c["window"], causal=c["causal"],
                                         sinks=c["sinks"]))
        if c["op"] == "bwd":
            return list(swa.swa_attn_bwd(s["q"], s["k"], s["v"], s["o"], s["do"], s["lse"],
                                         c["window"], causal=c["causal"], sinks=c["sinks"]))
        cache = swa.SwaCache(s["k"], s["v"], s["k_scale"], s["v_scale"], s["weight"])
        window = c["window"] or s["table"].shape[1] * c["page"]
        if c["op"] == "shared":
            return list(swa.swa_cache_attn(s["q"], cache, s["table"], s["lens"], window,
                                           new=s["new"], sinks=c["sinks"],
                                           shared=c["prefix"] // c["page"]))
        o, lse = swa.swa_cache_attn(s["q"], cache, s["table"], s["lens"], window, new=s["new"],
                                    accumulate=c["acc"], sinks=c["sinks"])
        return [o, lse, s["weight"]] if c["acc"] else [o, lse]
    if c["op"] == "fwd":
        return list(_forward(s["q"], s["k"], s["v"], c))
    if c["op"] == "bwd":
        return _backward(s, c)
    if c["op"] == "shared":
        return _shared(s, c)
    return _token(s, c)


def _blocks(c):
    """Blocks of queries [i, z) with the keys that the window reaches, [lo, hi), and the sinks before
    those, which every query of the block sees."""
    off, W, step = c["Lk"] - c["Lq"], c["window"], 1024
    for i in range(0, c["Lq"], step):
        z = min(c["Lq"], i + step)
        lo = max(0, i + off - W + 1)
        hi = z + off if c["causal"] else min(c["Lk"], z + off + W - 1)
        yield i, z, lo, hi, min(c["sinks"], lo)


def _visible(c, i, z, lo, hi, device):
    at = torch.arange(i, z, device=device)[:, None] + c["Lk"] - c["Lq"]
    key = torch.arange(lo, hi, device=device)
    near = (at - key < c["window"]) | (key < c["sinks"])
    return near & (at - key >= (0 if c["causal"] else 1 - c["window"]))


def _scores(q, k, c, i, z, lo, hi, n):
    """Scaled scores [B, Hkv, G, z - i, n + hi - lo] of a block; -inf where a key is not visible."""
    B, Hkv, G, _, D = q.shape
    x = q[:, :, :, i:z].reshape(B, Hkv, G * (z - i), D)
    far = x @ k[:, :, :n].transpose(-1, -2) / math.sqrt(D)
    near = x @ k[:, :, lo:hi].transpose(-1, -2) / math.sqrt(D)
    near = near.view(B, Hkv, G, z - i, hi - lo)
    near = torch.where(_visible(c, i, z, lo, hi, q.device), near, -math.inf)
    return torch.cat([far.view(B, Hkv, G, z - i, n), near], -1)


def _forward(q, k, v, c):
    B, Hq, Lq, D = q.shape
    Hkv, G = k.shape[1], Hq // k.shape[1]
    qf, kf, vf = q.float().view(B, Hkv, G, Lq, D), k.float(), v.float()
    o = torch.empty((B, Hkv, G, Lq, D), dtype=q.dtype, device=q.device)
    lse = torch.empty((B, Hkv, G, Lq), dtype=torch.float32, device=q.device)
    for i, z, lo, hi, n in _blocks(c):
        x = _scores(qf, kf, c, i, z, lo, hi, n)
        top = x.amax(-1, keepdim=True)
        p = torch.exp(x - top)
        total = p.sum(-1, keepdim=True)
        lse[:, :, :, i:z] = (top + torch.log(total)).squeeze(-1)
        p = (p / total).view(B, Hkv, G * (z - i), n + hi - lo)
        y = p[..., :n] @ vf[:, :, :n] + p[..., n:] @ vf[:, :, lo:hi]
        o[:, :, :, i:z] = y.view(B, Hkv, G, z - i, D).to(q.dtype)
    return o.view(B, Hq, Lq, D), lse.view(B, Hq, Lq)


def _backward(s, c):
    q, k, v = s["q"], s["k"], s["v"]
    B, Hq, Lq, D = q.shape
    Hkv, G = k.shape[1], Hq // k.shape[1]
    qf, do = q.float().view(B, Hkv, G, Lq, D), s["do"].float().view(B, Hkv, G, Lq, D)
    kf, vf = k.float(), v.float()
    delta = (do * s["o"].float().view_as(do)).sum(-1, keepdim=True)
    lse = s["lse"].view(B, Hkv, G, Lq, 1)
    dq = torch.empty((B, Hkv, G, Lq, D), dtype=q.dtype, device=q.device)
    dk, dv = torch.zeros_like(kf), torch.zeros_like(vf)
    scale = 1 / math.sqrt(D)
    for i, z, lo, hi, n in _blocks(c):
        rows = G * (z - i)
        p = torch.exp(_scores(qf, kf, c, i, z, lo, hi, n) - lse[:, :, :, i:z])
        g = do[:, :, :, i:z].reshape(B, Hkv, rows, D)
        dp = torch.cat([g @ vf[:, :, :n].transpose(-1, -2), g @ vf[:, :, lo:hi].transpose(-1, -2)],
                       -1).view_as(p)
        ds = (p * (dp - delta[:, :, :, i:z]) * scale).view(B, Hkv, rows, n + hi - lo)
        p = p.view_as(ds)
        y = ds[..., :n] @ kf[:, :, :n] + ds[..., n:] @ kf[:, :, lo:hi]
        dq[:, :, :, i:z] = y.view(B, Hkv, G, z - i, D).to(q.dtype)
        x = qf[:, :, :, i:z].reshape(B, Hkv, rows, D)
        dk[:, :, :n] += ds[..., :n].transpose(-1, -2) @ x
        dk[:, :, lo:hi] += ds[..., n:].transpose(-1, -2) @ x
        dv[:, :, :n] += p[..., :n].transpose(-1, -2) @ g
        dv[:, :, lo:hi] += p[..., n:].transpose(-1, -2) @ g
    return [dq.view(B, Hq, Lq, D), dk.to(k.dtype), dv.to(v.dtype)]


def _take(s, name, pages):
    """Values of a pool's pages [B, n] as tokens [B, Hkv, n page, D]."""
    x = s[name].view(torch.uint8)[pages].view(torch.float8_e4m3fn).float()
    x = (x * s[name + "_scale"][pages][..., None, None]).transpose(1, 2)
    return x.reshape(x.shape[0], x.shape[1], -1, x.shape[-1])


def _slots(s, c, first, n):
    """Slots and table entries of n pages of each sequence, from page first[b] on (entries behind the
    table's last repeat it: no query sees those slots)."""
    S = c["page"]
    i = first[:, None] + torch.arange(n, device="cuda")
    pages = s["table"].long().gather(1, i.clamp(max=s["table"].shape[1] - 1))
    return first[:, None] * S + torch.arange(n * S, device="cuda"), pages


def _sees(s, c, slots, W):
    """Whether query t of sequence b sees slots[b]: [B, T, L]."""
    t = torch.arange(c["T"], device="cuda")
    at = (s["lens"].long()[:, None] + t)[:, :, None]
    new = s["new"].long() if s["new"] is not None else torch.full_like(s["lens"], c["T"]).long()
    slots = slots[:, None]
    return ((slots <= at) & ((slots > at - W) | (slots < c["sinks"])) &
            (t[:, None] < new[:, None, None]))


def _softmax(x):
    """Weights of scores along the last dimension, and their log-sum-exp; a row of -inf gets none."""
    top = x.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(x - top)
    z = p.sum(-1, keepdim=True)
    return p / z.clamp(min=1e-30), torch.where(z > 0, top + torch.log(z), -math.inf)


def _token(s, c):
    B, Hkv, T, D, S = c["B"], c["Hkv"], c["T"], c["D"], c["page"]
    G, W = c["Hq"] // Hkv, c["window"]
    width = s["table"].shape[1]
    # the sinks' pages, then the window's; a slot in both counts in the second
    few = min(width, -(-c["sinks"] // S))
    first = (s["lens"].long() - W + 1).clamp(min=0) // S
    sink, near = _slots(s, c, torch.zeros_like(first), few), _slots(s, c, first,
                                                                    min(width, (W + T - 2) // S + 2))
    slots, pages = torch.cat([sink[0], near[0]], 1), torch.cat([sink[1], near[1]], 1)
    real = torch.cat([sink[0] < first[:, None] * S, near[0] < width * S], 1)
    sees = _sees(s, c, slots, W) & real[:, None]
    q = s["q"].float().view(B, Hkv, G * T, D)
    x = q @ _take(s, "k", pages).transpose(-1, -2) / math.sqrt(D)
    x = torch.where(sees[:, None, None], x.view(B, Hkv, G, T, -1), -math.inf).view_as(x)
    p, lse = _softmax(x)
    o = (p @ _take(s, "v", pages)).view(B, c["Hq"], T, D).to(s["q"].dtype)
    lse = lse.view(B, c["Hq"], T)
    if not c["acc"]:
        return [o, lse]
    add = p.sum(2).view(B, Hkv, -1, S).transpose(1, 2)
    s["weight"].index_put_((pages,), add, accumulate=True)
    return [o, lse, s["weight"]]


def _shared(s, c):
    B, Hkv, T, D, S, P = c["B"], c["Hkv"], c["T"], c["D"], c["page"], c["prefix"]
    G, common = c["Hq"] // Hkv, P // S
    W = c["window"] or 1 << 30
    q = s["q"].float().view(B, Hkv, G * T, D)

    def masked(x, slots):
        sees = _sees(s, c, slots, W)[:, None, None]
        return torch.where(sees, x.view(B, Hkv, G, T, -1), -math.inf).view_as(x)

    # the prefix for all sequences at once
    pages = s["table"][:1, :common].long()
    k, v = _take(s, "k", pages)[0], _take(s, "v", pages)[0]
    rows = q.transpose(0, 1).reshape(Hkv, B * G * T, D)
    far = (rows @ k.transpose(-1, -2)).view(Hkv, B, G * T, P).transpose(0, 1) / math.sqrt(D)
    far = masked(far, torch.arange(P, device="cuda").expand(B, P))
    # what follows it, for each
    slots, pages = _slots(s, c, torch.full_like(s["lens"], common).long(),
                          s["table"].shape[1] - common)
    near = masked(q @ _take(s, "k", pages).transpose(-1, -2) / math.sqrt(D), slots)
    p, lse = _softmax(torch.cat([far, near], -1))
    o = p[..., P:] @ _take(s, "v", pages)
    y = p[..., :P].transpose(0, 1).reshape(Hkv, B * G * T, P) @ v
    o += y.view(Hkv, B, G * T, D).transpose(0, 1)
    return [o.view(B, c["Hq"], T, D).to(s["q"].dtype), lse.view(B, c["Hq"], T)]


# ---- the definitions in 64 bits ----------------------------------------------------------------

def exact(case, seed):
    c, s = dict(case), prepare(case, seed)
    if c["op"] in ("fwd", "bwd"):
        return _exact_training(c, s)
    lens, new = _lengths(c)
    B, Hkv, T, D, S = c["B"], c["Hkv"], c["T"], c["D"], c["page"]
    G, W = c["Hq"] // Hkv, c["window"] or 1 << 30
    k, v = s["k"].double(), s["v"].double()
    ks, vs, table = s["k_scale"].double(), s["v_scale"].double(), s["table"].long()
    w = s["weight"].double() if c.get("acc") else None
    o = torch.zeros((B, c["Hq"], T, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, c["Hq"], T), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        for t in range(new[b]):
            p = lens[b] + t
            at = torch.arange(p + 1, device="cuda")
            at = at[(at > p - W) | (at < c["sinks"])]
            page = table[b, at // S]
            for h in range(Hkv):
                key = k[page, h, at % S] * ks[page, h, None]
                x = s["q"][b, h * G:(h + 1) * G, t].double() @ key.T / math.sqrt(D)
                z = torch.logsumexp(x, -1)
                e = torch.exp(x - z[:, None])
                o[b, h * G:(h + 1) * G, t] = e @ (v[page, h, at % S] * vs[page, h, None])
                lse[b, h * G:(h + 1) * G, t] = z
                if w is not None:
                    w[page, h, at % S] += e.sum(0)
    return [o, lse] if w is None else [o, lse, w]


def _exact_training(c, s):
    B, Hq, Lq, Lk, D, W = c["B"], c["Hq"], c["Lq"], c["Lk"], c["D"], c["window"]
    G, back = Hq // c["Hkv"], c["op"] == "bwd"
    if (min(Lk, 2 * W + 512 + c["sinks"]) * Lq * B * Hq * D * (5 if back else 2)) > 1 << 43:
        return None
    new = lambda *shape: torch.zeros(shape, dtype=torch.float64, device="cuda")  # noqa: E731
    o, lse, dq = new(B, Hq, Lq, D), new(B, Hq, Lq), new(B, Hq, Lq, D)
    dk, dv = new(B, c["Hkv"], Lk, D), new(B, c["Hkv"], Lk, D)
    for a in range(0, Lq, 512):
        pos = torch.arange(a, min(Lq, a + 512), device="cuda") + Lk - Lq
        key = torch.arange(Lk, device="cuda")
        key = key[(key < c["sinks"]) | ((key > int(pos[0]) - W) & (key < int(pos[-1]) + W))]
        d = pos[:, None] - key
        see = ((d < W) | (key < c["sinks"])) & (d >= 0 if c["causal"] else d > -W)
        for b in range(B):
            for h in range(Hq):
                q = s["q"][b, h, a:a + 512].double()
                k, v = s["k"][b, h // G, key].double(), s["v"][b, h // G, key].double()
                x = torch.where(see, q @ k.T / math.sqrt(D), -math.inf)
                if not back:
                    z = torch.logsumexp(x, -1)
                    lse[b, h, a:a + 512] = z
                    o[b, h, a:a + 512] = torch.exp(x - z[:, None]) @ v
                    continue
                e = torch.exp(x - s["lse"][b, h, a:a + 512, None].double())
                g = s["do"][b, h, a:a + 512].double()
                t = (g * s["o"][b, h, a:a + 512].double()).sum(-1, keepdim=True)
                y = e * (g @ v.T - t) / math.sqrt(D)
                dq[b, h, a:a + 512] = y @ k
                dk[b, h // G].index_add_(0, key, y.T @ q)
                dv[b, h // G].index_add_(0, key, e.T @ g)
    return [dq, dk, dv] if back else [o, lse]
