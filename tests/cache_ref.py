"""Plain 64-bit forms of the cache operators, token by token, for the tests of swa_cache_* and
swa_attn_key_weights.  A pool is a dict of CPU tensors in float64 (codes as the values they stand
for); nothing here uses the library."""
import math

import torch

E4M3_NAN = 0x7F


def e4m3_round(y):
    """Nearest e4m3 value, ties to even, for |y| <= 448 (NaN stays NaN)."""
    _, e = torch.frexp(y)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return torch.round(y / step) * step


def pool_of(cache):
    """float64 copies of a SwaCache's tensors on the CPU."""
    def codes(t):
        return t.view(torch.uint8).cpu().view(torch.float8_e4m3fn).float().double()

    return {"k": codes(cache.k), "v": codes(cache.v), "k_scale": cache.k_scale.cpu().double(),
            "v_scale": cache.v_scale.cpu().double(),
            "weight": None if cache.weight is None else cache.weight.cpu().double()}


def scale_for(amax):
    """Least 2^e, -48 <= e <= 40, with amax <= 448 2^e."""
    e = -48
    while e < 40 and amax > 448 * 2.0**e:
        e += 1
    return 2.0**e


def append(pool, table, lens, k, v, new=None, weight=None):
    B, H, T, D = k.shape
    S = pool["k"].shape[2]
    k, v = k.cpu().double(), v.cpu().double()
    for b in range(B):
        n = T if new is None else int(new[b])
        for h in range(H):
            at = int(lens[b])
            end = at + n
            while at < end:
                first = at - at % S
                stop = min(first + S, end)
                page = int(table[b, at // S])
                a, z, i = at - first, stop - first, at - int(lens[b])
                nk, nv = k[b, h, i:i + stop - at], v[b, h, i:i + stop - at]
                bad = ~((nk.abs() <= 448 * 2.0**40).all(-1) & (nv.abs() <= 448 * 2.0**40).all(-1))
                for name, x in (("k", nk), ("v", nv)):
                    fine = x[~bad]
                    now = scale_for(float(fine.abs().max()) if fine.numel() else 0.0)
                    if a:
                        old = float(pool[name + "_scale"][page, h])
                        now = max(now, old)
                        pool[name][page, h, :a] = e4m3_round(pool[name][page, h, :a] * (old / now))
                    pool[name + "_scale"][page, h] = now
                    y = torch.zeros_like(x)
                    y[~bad] = e4m3_round(fine / now)
                    if name == "k":
                        y[bad] = math.nan
                    pool[name][page, h, a:z] = y
                if pool["weight"] is not None:
                    pool["weight"][page, h, a:z] = \
                        0 if weight is None else weight[b, h, i:i + stop - at].cpu().double()
                at = stop


def tokens(pool, table, b, h, slots):
    """(k, v, (page, row)) of the given slots of sequence b, head h, in float64."""
    S = pool["k"].shape[2]
    page = torch.tensor([int(table[b, s // S]) for s in slots], dtype=torch.long)
    row = torch.tensor([s % S for s in slots], dtype=torch.long)
    k = pool["k"][page, h, row] * pool["k_scale"][page, h, None]
    v = pool["v"][page, h, row] * pool["v_scale"][page, h, None]
    return k, v, (page, row)


def attn(pool, table, lens, q, window, scale=None, new=None, accumulate=False):
    """(o, lse, tolerance of o, tolerance of lse, tolerance of the weights added).

    Tolerances, from the arithmetic the kernels may use: a score is an fp32 sum of D products
    (relative 2^-24 each step, and a rounding of the scaled score), so its error is at most
    es = (D + 8) 2^-24 scale <|q|, |k|>, plus the exponential's 2^-21; p is rounded to fp16 as an
    operand (2^-11, or 2^-25 where it is subnormal); o is rounded once to its type."""
    B, Hq, T, D = q.shape
    H = pool["k"].shape[1]
    G = Hq // H
    scale = 1 / math.sqrt(D) if scale is None else scale
    qd = q.cpu().double()
    o = torch.zeros((B, Hq, T, D), dtype=torch.float64)
    lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64)
    to, tl = torch.zeros_like(o), torch.zeros_like(lse)
    wt = None if pool["weight"] is None else torch.zeros_like(pool["weight"])
    half = torch.finfo(q.dtype).eps / 2
    for b in range(B):
        n = T if new is None else int(new[b])
        if n == 0:
            continue
        L = int(lens[b])
        base = max(0, L - window + 1)
        slots = range(base, L + n)
        for h in range(H):
            k, v, (page, row) = tokens(pool, table, b, h, slots)
            for t in range(n):
                lo, hi = max(0, L + t - window + 1) - base, L + t + 1 - base
                qq = qd[b, h * G:(h + 1) * G, t]
                kk, vv = k[lo:hi], v[lo:hi]
                x = qq @ kk.T * scale
                es = ((D + 8) * 2.0**-24 * (qq.abs() @ kk.abs().T * scale)).amax(-1, keepdim=True)
                es = es + 2.0**-21
                z = torch.logsumexp(x, -1, keepdim=True)
                p = torch.exp(x - z)
                o[b, h * G:(h + 1) * G, t] = r = p @ vv
                mag = p @ vv.abs()
                to[b, h * G:(h + 1) * G, t] = mag * (2.0**-11 + 2 * es) + \
                    2.0**-25 * vv.abs().sum(0) + 1.01 * half * r.abs() + \
                    (2.0**-25 if q.dtype == torch.float16 else 0.0)
                lse[b, h * G:(h + 1) * G, t] = z[:, 0]
                tl[b, h * G:(h + 1) * G, t] = es[:, 0] + 2.0**-21 * (1 + z[:, 0].abs())
                if accumulate:
                    pool["weight"][page[lo:hi], h, row[lo:hi]] += p.sum(0)
                    wt[page[lo:hi], h, row[lo:hi]] += (p * (2 * es + 2.0**-20)).sum(0)
    if accumulate:
        wt = wt + 2.0**-22 * pool["weight"].abs()
    return o, lse, to, tl, wt


def evict(pool, table, lens, dst, budget, recent):
    """(kept [B,H,budget], lens_out); the pool's destination pages are written in place."""
    B = table.shape[0]
    H, S = pool["k"].shape[1], pool["k"].shape[2]
    kept = torch.full((B, H, budget), -1, dtype=torch.int32)
    out = torch.zeros(B, dtype=torch.int32)
    for b in range(B):
        L = int(lens[b])
        m = min(L, budget)
        out[b] = m
        for h in range(H):
            if L <= budget:
                stay = list(range(L))
            else:
                w = [float(pool["weight"][int(table[b, s // S]), h, s % S]) for s in range(L - recent)]
                order = sorted(range(L - recent),
                               key=lambda s: (-math.inf if math.isnan(w[s]) else -w[s],
                                              0 if math.isnan(w[s]) else 1, s))
                stay = sorted(order[:budget - recent]) + list(range(L - recent, L))
            kept[b, h, :m] = torch.tensor(stay, dtype=torch.int32)
            for j in range(0, m, S):
                some = stay[j:j + S]
                to = int(dst[b, j // S])
                page = torch.tensor([int(table[b, s // S]) for s in some], dtype=torch.long)
                row = torch.tensor([s % S for s in some], dtype=torch.long)
                z = len(some)
                pool["weight"][to, h, :z] = pool["weight"][page, h, row]
                for name in ("k", "v"):
                    was = pool[name + "_scale"][page, h]
                    now = was.max()
                    pool[name][to, h, :z] = e4m3_round(pool[name][page, h, row] *
                                                       (was / now)[:, None])
                    pool[name + "_scale"][to, h] = now
    return kept, out


def key_weights(q, k, lse, window, scale=None, causal=True):
    """(w, tolerance): a score's fp32 sum of D products, as in attn(), and the sum over rows."""
    B, Hq, Lq, D = q.shape
    H, Lk = k.shape[1], k.shape[2]
    G = Hq // H
    scale = 1 / math.sqrt(D) if scale is None else scale
    qd = q.cpu().double().view(B, H, G * Lq, D)
    kd = k.cpu().double()
    x = qd @ kd.transpose(-1, -2) * scale
    es = (D + 8) * 2.0**-24 * (qd.abs() @ kd.abs().transpose(-1, -2) * scale) + 2.0**-21
    d = torch.arange(Lq)[:, None] + (Lk - Lq) - torch.arange(Lk)
    see = (d < window) & ((d >= 0) if causal else (d > -window))
    see = see.repeat(G, 1)
    z = lse.cpu().double().view(B, H, G * Lq, 1)
    es = es + 2.0**-22 * z.abs()
    p = torch.where(see, torch.exp(x - z), torch.zeros((), dtype=torch.float64))
    w = p.sum(2)
    # rows are added in fp32, at most G Lq of them in one chain
    tol = (p * 2 * es).sum(2) + (G * Lq) * 2.0**-24 * w + 1e-30
    return w, tol
