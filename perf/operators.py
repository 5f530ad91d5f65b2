"""The serving operators beside the training attention, as cases that can be timed and checked.

Four operators work together when a model trained with this library's attention answers with it:

  append       new keys and values go into a paged cache held in 8 bits (e4m3), one power-of-two
               scale for each page (a block of tokens) and kv head
  attn         attention of one token, or of a few that are verified at once, over that cache,
               optionally adding the weight that each cached token received to a running sum
  evict        the cache is cut to a budget: the most recent tokens stay, and of the others those
               with the largest accumulated weight, moved to pages of their own
  key_weights  the weight that each key of a whole prompt received, from q, k and the forward's
               log-sum-exp: what a prompt's tokens enter the cache with

`run` computes each in plain torch operations in 32 bits, or, with `own`, by the library's calls.
"""
import math
import random

import torch

own = False

SCALE_MIN, SCALE_MAX = -48, 40  # exponents of a block's scale
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # A decode step's new token of 16 sequences, somewhere inside a page each: latency.
        dict(name="append token", op="append", B=16, Hkv=16, D=128, page=64, T=1, longest=8192,
             ragged=False, weight=False, dtype="bf16", spread=1),
        # A whole prompt of the longest example's length into an empty cache, with the weights
        # that its tokens already received.
        dict(name="append prompt", op="append", B=1, Hkv=16, D=128, page=64, T=30553, longest=0,
             ragged=False, weight=True, dtype="bf16", spread=2),
        # Chunks of four sequences that begin and end inside pages, of unequal lengths.
        dict(name="append chunk d256", op="append", B=4, Hkv=16, D=256, page=32, T=517,
             longest=4000, ragged=True, weight=False, dtype="fp16", spread=3),
        # One user, one token, a sliding layer: the smallest call of a decode loop.
        dict(name="attn token window", op="attn", B=1, Hq=32, Hkv=16, D=128, page=64, T=1,
             shortest=32768, longest=32768, window=1024, ragged=False, acc=False, dtype="bf16",
             spread=4),
        # A full layer of a batch server: contexts from short to long, weights accumulated.
        dict(name="attn batch ragged", op="attn", B=64, Hq=32, Hkv=8, D=128, page=64, T=1,
             shortest=1, longest=16384, window=0, ragged=False, acc=True, dtype="bf16", spread=5),
        # Long documents in full layers: the cache's bytes are everything.
        dict(name="attn long", op="attn", B=8, Hq=32, Hkv=16, D=128, page=128, T=1,
             shortest=120000, longest=131072, window=0, ragged=False, acc=False, dtype="bf16",
             spread=6),
        # A few drafted tokens of each sequence verified at once in sliding layers, wide heads.
        dict(name="attn verify d256", op="attn", B=12, Hq=32, Hkv=16, D=256, page=32, T=5,
             shortest=700, longest=30553, window=1024, ragged=True, acc=False, dtype="fp16",
             spread=7),
        # After one long prompt: a full layer's cache cut to an eighth.
        dict(name="evict prompt", op="evict", B=1, Hkv=16, D=128, page=64, shortest=30553,
             longest=30553, budget=4096, recent=512, spread=8),
        # A batch that outgrew its budget at different times.
        dict(name="evict batch", op="evict", B=32, Hkv=8, D=128, page=64, shortest=100,
             longest=8192, budget=2000, recent=250, spread=9),
        # The long sliding-window layer's prompt.
        dict(name="key weights window", op="key_weights", B=1, Hq=32, Hkv=16, Lq=32768, Lk=32768,
             D=128, window=1024, dtype="bf16"),
        # The causal prompt of a full layer, four query heads to a kv head.
        dict(name="key weights causal", op="key_weights", B=1, Hq=32, Hkv=8, Lq=8192, Lk=8192,
             D=128, window=8192, dtype="bf16"),
        # A short suffix of a short prompt, narrow heads.
        dict(name="key weights suffix", op="key_weights", B=2, Hq=4, Hkv=2, Lq=255, Lk=1000, D=64,
             window=64, dtype="fp16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "evict", "key_weights"])
    D = rng.choice([64, 128, 128, 256])
    page = rng.choice([32, 64, 64, 128])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    spread = rng.randrange(1000)
    if op == "append":
        T = _log_int(rng, 1, 20000)
        B = _log_int(rng, 1, max(1, min(64, 30553 * 16 * 128 // (T * Hkv * D))))
        return dict(op=op, B=B, Hkv=Hkv, D=D, page=page, T=T, longest=_log_int(rng, 1, 8192),
                    ragged=rng.random() < 0.5, weight=rng.random() < 0.5,
                    dtype=rng.choice(["bf16", "fp16", "fp32"]), spread=spread)
    if op == "attn":
        T = rng.choice([1, 1, 1, 2, 3, 5, 8])
        G = rng.choice([1, 2, 4, 7, 8])
        longest = _log_int(rng, 16, 65536)
        B = _log_int(rng, 1, max(1, min(96, (1 << 31) // (longest * Hkv * D * 2))))
        return dict(op=op, B=B, Hq=G * Hkv, Hkv=Hkv, D=D, page=page, T=T,
                    shortest=_log_int(rng, 1, longest), longest=longest,
                    window=rng.choice([0, 0, _log_int(rng, 1, 4096)]),
                    ragged=T > 1 and rng.random() < 0.5, acc=rng.random() < 0.5,
                    dtype=rng.choice(["bf16", "fp16"]), spread=spread)
    if op == "evict":
        longest = _log_int(rng, 64, 65536)
        B = _log_int(rng, 1, max(1, min(32, (1 << 28) // (longest * Hkv * D))))
        budget = _log_int(rng, 16, max(16, longest // 2))
        return dict(op=op, B=B, Hkv=Hkv, D=D, page=page, shortest=_log_int(rng, 1, longest),
                    longest=longest, budget=budget, recent=rng.randrange(budget + 1),
                    spread=spread)
    Lk = _log_int(rng, 64, 16384)
    Lq = Lk if rng.random() < 0.6 else _log_int(rng, 1, Lk)
    window = Lk if rng.random() < 0.3 and Lk <= 8192 else _log_int(rng, 1, min(Lk, 2048))
    G = rng.choice([1, 2, 4])
    Hkv = min(Hkv, 8)
    return dict(op=op, B=rng.choice([1, 1, 2]) if Lk <= 4096 else 1, Hq=G * Hkv, Hkv=Hkv, Lq=Lq,
                Lk=Lk, D=D, window=window, dtype=rng.choice(["bf16", "fp16"]))


# ---- sizes that follow from a case alone -------------------------------------------------------

def _lengths(c):
    """(tokens in the cache before the call, new tokens) of each sequence."""
    r = random.Random(c["spread"])
    lo, hi = c.get("shortest", 0), c.get("longest", 0)
    T = c.get("T", 0)
    lens = [r.randint(lo, hi) for _ in range(c["B"])]
    if c["op"] == "attn":  # the new tokens are the last of these
        lens = [max(0, n - T) for n in lens]
    new = [r.randint(0, T) if c.get("ragged") else T for _ in range(c["B"])]
    return lens, new


def _pages(c):
    """Pages of each sequence's table."""
    lens, _ = _lengths(c)
    return -(-(max(lens) + max(1, c.get("T", 0))) // c["page"])


def _pairs(Lq, Lk, W):
    """Visible (query, key) pairs of one head: query i sees keys i + Lk - Lq - W + 1 .. i + Lk - Lq."""
    first = Lk - Lq + 1  # keys that query 0 sees without a window
    cut = min(Lq, max(0, W - first + 1))  # queries that see fewer than W
    return cut * first + cut * (cut - 1) // 2 + (Lq - cut) * W if W < Lk else \
        Lq * first + Lq * (Lq - 1) // 2


def work(case):
    c = case
    if c["op"] == "key_weights":
        es = 2
        n = _pairs(c["Lq"], c["Lk"], c["window"]) * c["B"] * c["Hq"]
        return {"bytes": c["B"] * (c["Hq"] * c["Lq"] * (c["D"] * es + 4) +
                                   c["Hkv"] * c["Lk"] * (c["D"] * es + 4)),
                "flops": 2 * c["D"] * n}
    lens, new = _lengths(c)
    if c["op"] == "append":
        es = 4 if c["dtype"] == "fp32" else 2
        n = sum(new) * c["Hkv"]
        blocks = sum(-(-(a + m) // c["page"]) - a // c["page"] for a, m in zip(lens, new) if m)
        return {"bytes": n * (2 * c["D"] * (es + 1) + 4 + 4 * c["weight"]) +
                8 * blocks * c["Hkv"] + 8 * c["B"],
                "flops": 0}
    if c["op"] == "evict":
        kept = sum(min(n, c["budget"]) for n in lens) * c["Hkv"]
        return {"bytes": 4 * sum(lens) * c["Hkv"] + kept * (4 * c["D"] + 8) +
                4 * c["B"] * c["Hkv"] * c["budget"], "flops": 0}
    W = c["window"] or 1 << 30
    keys = pairs = 0
    for a, m in zip(lens, new):
        if m:
            keys += a + m - max(0, a + 1 - W)
            pairs += sum(min(a + t + 1, W) for t in range(m))
    rows = c["B"] * c["Hq"] * c["T"]
    return {"bytes": keys * c["Hkv"] * (2 * c["D"] + 8 * c["acc"] + 8 / c["page"]) +
            rows * (4 * c["D"] + 4),
            "flops": 4 * c["D"] * pairs * c["Hq"]}


# ---- inputs ------------------------------------------------------------------------------------

def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[c.get("dtype", "bf16")]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    s = {"case": c}
    if c["op"] == "key_weights":
        s["q"] = normal(c["B"], c["Hq"], c["Lq"], c["D"]).to(dt)
        s["k"] = normal(c["B"], c["Hkv"], c["Lk"], c["D"]).to(dt)
        s["lse"] = _banded(s["q"], s["k"], c["window"], None)
        return s
    lens, new = _lengths(c)
    n = _pages(c)
    out = -(-c["budget"] // c["page"]) if c["op"] == "evict" else 0
    total = c["B"] * (n + out) + 1  # the last page belongs to nobody
    page, D, Hkv, B = c["page"], c["D"], c["Hkv"], c["B"]
    # Codes as quantised activations have them: nearly normal, the largest of a block near 448.
    for name in ("k", "v"):
        s[name] = (normal(total, Hkv, page, D) * 100).clamp_(-448, 448).to(torch.float8_e4m3fn)
        s[name + "_scale"] = torch.exp2(torch.randint(-8, -5, (total, Hkv), generator=g,
                                                      device="cuda").float())
    # Attention weights are very unequal: a few tokens hold most of them.
    s["weight"] = torch.exp(2 * normal(total, Hkv, page))
    order = torch.randperm(total - 1, generator=g, device="cuda").to(torch.int32)
    s["table"] = order[:B * n].view(B, n).contiguous()
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if c["op"] == "evict":
        s["dst"] = order[B * n:].view(B, out).contiguous()
        return s
    s["new"] = torch.tensor(new, dtype=torch.int32, device="cuda") if c["ragged"] else None
    T = c["T"]
    if c["op"] == "append":
        for name in ("new_k", "new_v"):
            s[name] = (normal(B, Hkv, T, D) * torch.exp(normal(B, Hkv, 1, 1))).to(dt)
        s["new_weight"] = torch.exp(2 * normal(B, Hkv, T)) if c["weight"] else None
    else:
        s["q"] = normal(B, c["Hq"], T, D).to(dt)
    return s


# ---- one pass ----------------------------------------------------------------------------------

def run(state):
    s, c = state, state["case"]
    if c["op"] == "key_weights":
        if own:
            import sliding_window_flash_gb300 as swa
            return swa.swa_attn_key_weights(s["q"], s["k"], s["lse"], c["window"])
        return _banded(s["q"], s["k"], c["window"], s["lse"])
    if own:
        import sliding_window_flash_gb300 as swa
        cache = swa.SwaCache(s["k"], s["v"], s["k_scale"], s["v_scale"], s["weight"])
        if c["op"] == "append":
            swa.swa_cache_append(cache, s["table"], s["lens"], s["new_k"], s["new_v"],
                                 new=s["new"], weight=s["new_weight"])
            return _pool(s)
        if c["op"] == "evict":
            kept, lens = swa.swa_cache_evict(cache, s["table"], s["lens"], s["dst"], c["budget"],
                                             c["recent"])
            return [kept, lens, _pool(s)]
        o, lse = swa.swa_cache_attn(s["q"], cache, s["table"], s["lens"],
                                    c["window"] or s["table"].shape[1] * c["page"],
                                    new=s["new"], accumulate=c["acc"])
    elif c["op"] == "append":
        _append(s)
        return _pool(s)
    elif c["op"] == "evict":
        kept, lens = _evict(s)
        return [kept, lens, _pool(s)]
    else:
        o, lse = _attn(s)
    return [o, lse, s["weight"]] if c["acc"] else [o, lse]


def _pool(s):
    """The whole cache: e4m3 values in units of their block's scale, the scales, the weights."""
    return [s["k"], s["v"], s["k_scale"], s["v_scale"], s["weight"]]


def _take(pool, pages):
    """pool [P, Hkv, page, ...] at pages [B, n], as [B, n, Hkv, page, ...] (8-bit pools as fp32)."""
    if pool.dtype == torch.float8_e4m3fn:
        return pool.view(torch.uint8)[pages].view(torch.float8_e4m3fn).float()
    return pool[pages]


def _scale_for(amax):
    """The least power of two, in the range allowed, that brings amax to at most 448."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    return torch.exp2(torch.where(amax > 0, e, SCALE_MIN).clamp(SCALE_MIN, SCALE_MAX).float())


def _append(s):
    c = s["case"]
    S, T, D = c["page"], c["T"], c["D"]
    lens = s["lens"].long()
    new = s["new"].long() if s["new"] is not None else torch.full_like(lens, T)
    n = (S + T - 2) // S + 1  # pages that T tokens touch at most
    first = lens // S
    pos = first[:, None] * S + torch.arange(n * S, device="cuda")
    src = pos - lens[:, None]
    fresh = ((src >= 0) & (src < new[:, None])).view(-1, n, 1, S)
    older = (src < 0).view(-1, n, 1, S)
    at = src.clamp(0, T - 1)
    touched = fresh.any(-1).squeeze(-1)
    idx = (first[:, None] + torch.arange(n, device="cuda")).clamp(max=s["table"].shape[1] - 1)
    nobody = s["weight"].shape[0] - 1
    pages = torch.where(touched, s["table"].long().gather(1, idx), nobody)
    for name in ("k", "v"):
        x = s["new_" + name].float().gather(2, at[:, None, :, None].expand(-1, c["Hkv"], -1, D))
        x = x.view(-1, c["Hkv"], n, S, D).transpose(1, 2)
        old, was = _take(s[name], pages), s[name + "_scale"][pages]
        need = _scale_for(torch.where(fresh[..., None], x.abs(), 0.0).amax((-1, -2)))
        now = torch.where(older.any(-1), torch.maximum(was, need), need)
        codes = torch.where(fresh[..., None], x / now[..., None, None],
                            torch.where(older[..., None], old * (was / now)[..., None, None], old))
        codes = codes.to(torch.float8_e4m3fn)
        s[name].view(torch.uint8)[pages] = codes.view(torch.uint8)
        s[name + "_scale"][pages] = torch.where(touched[..., None], now, was)
    w = torch.zeros((), device="cuda")
    if s["new_weight"] is not None:
        w = s["new_weight"].gather(2, at[:, None].expand(-1, c["Hkv"], -1))
        w = w.view(-1, c["Hkv"], n, S).transpose(1, 2)
    s["weight"][pages] = torch.where(fresh, w, s["weight"][pages])


def _attn(s):
    c = s["case"]
    B, Hkv, T, D, S = c["B"], c["Hkv"], c["T"], c["D"], c["page"]
    G = c["Hq"] // Hkv
    width = s["table"].shape[1]
    W = c["window"] or width * S
    lens = s["lens"].long()
    new = s["new"].long() if s["new"] is not None else torch.full_like(lens, T)
    first = (lens - W + 1).clamp(min=0) // S
    n = min(width, (W + T - 2) // S + 2)
    pos = first[:, None] * S + torch.arange(n * S, device="cuda")  # [B, L]
    idx = (first[:, None] + torch.arange(n, device="cuda")).clamp(max=width - 1)
    pages = s["table"].long().gather(1, idx)

    def tokens(name):
        x = _take(s[name], pages) * s[name + "_scale"][pages][..., None, None]
        return x.transpose(1, 2).reshape(B, Hkv, n * S, D)

    t = torch.arange(T, device="cuda")
    at = (lens[:, None] + t)[:, :, None]  # [B, T, 1]
    seen = (pos[:, None] <= at) & (pos[:, None] > at - W) & (t[:, None] < new[:, None, None])
    seen = seen[:, None, None].expand(B, Hkv, G, T, n * S).reshape(B, Hkv, G * T, n * S)
    q = s["q"].float().view(B, Hkv, G * T, D)
    x = (q @ tokens("k").transpose(-1, -2)) / math.sqrt(D)
    x = torch.where(seen, x, -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(x - m)
    z = p.sum(-1, keepdim=True)
    lse = torch.where(z > 0, m + torch.log(z), -math.inf)
    p = p / z.clamp(min=1e-30)
    o = p @ tokens("v")
    if c["acc"]:
        add = p.sum(2).view(B, Hkv, n, S).transpose(1, 2)
        s["weight"].index_put_((pages,), add, accumulate=True)
    return (o.view(B, c["Hq"], T, D).to(s["q"].dtype), lse.view(B, c["Hq"], T))


def _evict(s):
    c = s["case"]
    B, Hkv, S, D = c["B"], c["Hkv"], c["page"], c["D"]
    lens, pages = s["lens"].long(), s["table"].long()
    L, budget = pages.shape[1] * S, c["budget"]
    room = s["dst"].shape[1] * S
    pos = torch.arange(L, device="cuda")
    w = s["weight"][pages].transpose(1, 2).reshape(B, Hkv, L)
    held = lens[:, None, None]
    w = torch.where(pos >= held - c["recent"], math.inf, w)
    w = torch.where(pos < held, w, -math.inf)
    best = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :budget]
    kept = torch.where(best < held, best, L).sort(-1).values
    if kept.shape[-1] < room:
        kept = torch.nn.functional.pad(kept, (0, room - kept.shape[-1]), value=L)
    ok = (kept < held).view(B, Hkv, -1, S).transpose(1, 2)  # [B, n, Hkv, page]
    at = kept.clamp(max=L - 1)
    page = pages[torch.arange(B, device="cuda")[:, None, None], at // S]
    head = torch.arange(Hkv, device="cuda")[None, :, None]
    dst = s["dst"].long()
    for name in ("k", "v"):
        codes = s[name].view(torch.uint8)[page, head, at % S].view(torch.float8_e4m3fn).float()
        codes = codes.view(B, Hkv, -1, S, D).transpose(1, 2)
        was = s[name + "_scale"][page, head].view(B, Hkv, -1, S).transpose(1, 2)
        now = torch.where(ok, was, 0.0).amax(-1)
        some = now > 0
        now = torch.where(some, now, s[name + "_scale"][dst])
        codes = (codes * (was / now[..., None])[..., None]).to(torch.float8_e4m3fn)
        old = s[name].view(torch.uint8)[dst]
        s[name].view(torch.uint8)[dst] = torch.where(ok[..., None], codes.view(torch.uint8), old)
        s[name + "_scale"][dst] = now
    add = s["weight"][page, head, at % S].view(B, Hkv, -1, S).transpose(1, 2)
    s["weight"][dst] = torch.where(ok, add, s["weight"][dst])
    kept = torch.where(kept < held, kept, -1)[..., :budget]
    if kept.shape[-1] < budget:
        kept = torch.nn.functional.pad(kept, (0, budget - kept.shape[-1]), value=-1)
    return kept.to(torch.int32), lens.clamp(max=budget).to(torch.int32)


def _banded(q, k, window, lse):
    """Softmax over a causal window by blocks of keys as wide as the window: each row's
    log-sum-exp, or with `lse` the weight that each key receives from all the rows of its group."""
    B, Hq, Lq, D = q.shape
    Hkv, Lk = k.shape[1], k.shape[2]
    G = Hq // Hkv
    w = max(min(window, Lk), min(64, Lk))
    nb = -(-Lk // w)
    pad = torch.nn.functional.pad
    full = pad(q.float(), (0, 0, Lk - Lq, nb * w - Lk))  # queries at their key positions
    full = full.view(B, Hkv, G, nb, w, D)
    kb = pad(k.float(), (0, 0, 0, nb * w - Lk)).view(B, Hkv, 1, nb, w, D)
    i = torch.arange(nb * w, device=q.device).view(nb, w)
    real = (i >= Lk - Lq) & (i < Lk)

    def scores(shift):  # query block j + shift against key block j
        x = full[:, :, :, shift:] @ kb[:, :, :, :nb - shift].transpose(-1, -2) / math.sqrt(D)
        d = i[shift:, :, None] - i[:nb - shift, None, :]
        return x, (d >= 0) & (d < window) & real[shift:, :, None]

    if lse is None:
        z = torch.zeros((B, Hkv, G, nb, w), dtype=torch.float32, device=q.device)
        top = torch.full_like(z, -1e30)
        x, see = scores(0)
        x = torch.where(see, x, -math.inf)
        top = torch.maximum(top, x.amax(-1))
        y = None
        if nb > 1:
            y, see = scores(1)
            y = torch.where(see, y, -math.inf)
            top[:, :, :, 1:] = torch.maximum(top[:, :, :, 1:], y.amax(-1))
        z += torch.exp(x - top[..., None]).sum(-1)
        if y is not None:
            z[:, :, :, 1:] += torch.exp(y - top[:, :, :, 1:, :, None]).sum(-1)
        out = top + torch.log(z)
        return out.reshape(B, Hq, nb * w)[:, :, Lk - Lq:Lk].contiguous()
    base = pad(lse, (Lk - Lq, nb * w - Lk)).view(B, Hkv, G, nb, w, 1)
    x, see = scores(0)
    out = torch.where(see, torch.exp(x - base), 0.0).sum((2, -2))  # [B, Hkv, nb, w]
    if nb > 1:
        y, see = scores(1)
        out[:, :, :nb - 1] += torch.where(see, torch.exp(y - base[:, :, :, 1:]), 0.0).sum((2, -2))
    return out.reshape(B, Hkv, nb * w)[:, :, :Lk].contiguous()


# ---- the definitions in 64 bits ----------------------------------------------------------------

def _e4m3(y):
    """The nearest e4m3 value (ties to even) of numbers up to 448, by arithmetic."""
    _, e = torch.frexp(y)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return torch.round(y / step) * step


def exact(case, seed):
    c, s = dict(case), prepare(case, seed)
    if c["op"] == "key_weights":
        return _exact_key_weights(c, s)
    S, Hkv, B = c["page"], c["Hkv"], c["B"]
    lens, new = _lengths(c)
    k, v = s["k"].double(), s["v"].double()
    ks, vs, w = s["k_scale"].double(), s["v_scale"].double(), s["weight"].double()
    table = s["table"].long()
    if c["op"] == "append":
        for b in range(B):
            for first in range(lens[b] // S * S, lens[b] + new[b], S) if new[b] else ():
                page = int(table[b, first // S])
                lo, hi = max(first, lens[b]), min(first + S, lens[b] + new[b])
                a, z = lo - first, hi - first
                for pool, scale, x in ((k, ks, s["new_k"]), (v, vs, s["new_v"])):
                    x = x[b, :, lo - lens[b]:hi - lens[b]].double()
                    top = x.abs().amax((1, 2))
                    e = torch.ceil(torch.log2(top / 448)).clamp(SCALE_MIN, SCALE_MAX)
                    e = torch.where(top <= 448 * torch.exp2(e - 1), e - 1, e)
                    e = torch.where(top > 448 * torch.exp2(e), e + 1, e)
                    now = torch.exp2(e.clamp(SCALE_MIN, SCALE_MAX))
                    if a:
                        now = torch.maximum(now, scale[page])
                        pool[page, :, :a] = _e4m3(pool[page, :, :a] *
                                                  (scale[page] / now)[:, None, None])
                    scale[page] = now
                    pool[page, :, a:z] = _e4m3(x / now[:, None, None])
                given = s["new_weight"]
                w[page, :, a:z] = 0 if given is None else given[b, :, lo - lens[b]:hi - lens[b]]
        return [k, v, ks, vs, w]
    if c["op"] == "evict":
        budget, recent = c["budget"], c["recent"]
        kept = torch.full((B, Hkv, budget), -1, dtype=torch.int32, device="cuda")
        for b in range(B):
            n = lens[b]
            m = min(n, budget)
            at = torch.arange(n, device="cuda")
            page = table[b, at // S]
            keep = at.expand(Hkv, n)
            if n > budget:
                old = w[page, :, at % S].T[:, :n - recent]  # [Hkv, n - recent]
                best = torch.argsort(-old, dim=-1, stable=True)[:, :budget - recent]
                keep = torch.cat([best, at[n - recent:].expand(Hkv, recent)], 1).sort(-1).values
            kept[b, :, :m] = keep.to(torch.int32)
            head = torch.arange(Hkv, device="cuda")[:, None]
            src = page[keep]
            for j in range(0, m, S):
                to, z = int(s["dst"][b, j // S]), min(S, m - j)
                p, o = src[:, j:j + z], keep[:, j:j + z] % S
                w[to, :, :z] = w[p, head, o]
                for pool, scale in ((k, ks), (v, vs)):
                    one = scale[p, head]
                    now = one.amax(1)
                    x = pool[p, head, o] * (one / now[:, None])[..., None]
                    pool[to, :, :z] = _e4m3(x)
                    scale[to] = now
        return [kept, s["lens"].clamp(max=budget), [k, v, ks, vs, w]]
    T, D, G, W = c["T"], c["D"], c["Hq"] // Hkv, c["window"] or 1 << 30
    o = torch.zeros((B, c["Hq"], T, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, c["Hq"], T), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        for t in range(new[b]):
            at = torch.arange(max(0, lens[b] + t + 1 - W), lens[b] + t + 1, device="cuda")
            page = table[b, at // S]
            for h in range(Hkv):
                key = k[page, h, at % S] * ks[page, h, None]
                x = s["q"][b, h * G:(h + 1) * G, t].double() @ key.T / math.sqrt(D)
                z = torch.logsumexp(x, -1)
                p = torch.exp(x - z[:, None])
                o[b, h * G:(h + 1) * G, t] = p @ (v[page, h, at % S] * vs[page, h, None])
                lse[b, h * G:(h + 1) * G, t] = z
                if c["acc"]:
                    w[page, h, at % S] += p.sum(0)
    return [o, lse, w] if c["acc"] else [o, lse]


def _exact_key_weights(c, s):
    Lq, Lk, W, G = c["Lq"], c["Lk"], c["window"], c["Hq"] // c["Hkv"]
    if _pairs(Lq, Lk, W) * c["B"] * c["Hq"] * c["D"] > 1 << 38:
        return None
    out = torch.zeros((c["B"], c["Hkv"], Lk), dtype=torch.float64, device="cuda")
    off, step = Lk - Lq, 1024
    for b in range(c["B"]):
        for h in range(c["Hq"]):
            for i in range(0, Lq, step):
                z = min(Lq, i + step)
                lo, hi = max(0, i + off - W + 1), z + off
                x = s["q"][b, h, i:z].double() @ s["k"][b, h // G, lo:hi].double().T
                p = torch.exp(x / math.sqrt(c["D"]) - s["lse"][b, h, i:z, None].double())
                d = torch.arange(i, z, device="cuda")[:, None] + off - \
                    torch.arange(lo, hi, device="cuda")
                out[b, h // G, lo:hi] += torch.where((d >= 0) & (d < W), p, 0.0).sum(0)
    return out
