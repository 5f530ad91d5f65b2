"""The weights that a prompt's keys received, with sinks: key j counts the queries i (at position
i + Lk - Lq) with d = position - j >= 0 (two-sided: > -window) and d < window or j < sinks."""
import math

import pytest
import torch

BF16, FP16 = torch.bfloat16, torch.float16


def visible(Lq, Lk, window, sinks, causal, device="cuda"):
    d = torch.arange(Lq, device=device)[:, None] + (Lk - Lq) - torch.arange(Lk, device=device)
    near = (d < window) | (torch.arange(Lk, device=device) < sinks)
    return near & ((d >= 0) if causal else (d > -window))


def reference(q, k, lse, window, sinks, causal, scale=None):
    """(weights, tolerances) in 64 bits.  A score is an fp32 sum of D products, each step and the rounding of
    the scaled score 2^-24: es = (D + 8) 2^-24 scale <|q|, |k|> plus 2^-21 for the exponential and 2^-22 of
    the lse; rows are added in fp32, at most G Lq in one chain."""
    B, Hq, Lq, D = q.shape
    H, Lk = k.shape[1], k.shape[2]
    scale = 1 / math.sqrt(D) if scale is None else scale
    w, tol = (torch.zeros((B, H, Lk), dtype=torch.float64, device="cuda") for _ in range(2))
    see = visible(Lq, Lk, window, sinks, causal)
    for b in range(B):
        for h in range(Hq):
            g = h // (Hq // H)
            qd, kd, z = q[b, h].double(), k[b, g].double(), lse[b, h].double()[:, None]
            es = (D + 8) * 2.0**-24 * scale * (qd.abs() @ kd.abs().T) + 2.0**-21 + 2.0**-22 * z.abs()
            p = torch.where(see, torch.exp(qd @ kd.T * scale - z), 0.0)
            w[b, g] += p.sum(0)
            tol[b, g] += (p * 2 * es).sum(0)
    return w, tol + Hq // H * Lq * 2.0**-24 * w + 1e-30


def lse_of(q, k, window, sinks, causal, scale=None):
    G, scale = q.shape[1] // k.shape[1], 1 / math.sqrt(q.shape[3]) if scale is None else scale
    x = q.double() @ k.double().repeat_interleave(G, 1).mT * scale
    see = visible(q.shape[2], k.shape[2], window, sinks, causal)
    return torch.logsumexp(x.masked_fill(~see, -math.inf), -1).float()


def normal(g, *shape, dtype=BF16):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hq,H,Lq,Lk,D,window,sinks,causal,dtype", [
    (1, 1, 1, 1, 2, 64, 1, 1, True, BF16),
    (2, 4, 2, 255, 255, 64, 64, 4, True, FP16),
    (1, 2, 1, 300, 300, 128, 1, 300, True, BF16),       # every key a sink
    (1, 6, 2, 130, 1000, 128, 77, 129, True, FP16),     # queries a suffix
    (1, 4, 1, 700, 700, 256, 200, 1, True, BF16),
    (2, 2, 1, 129, 600, 256, 100, 257, True, FP16),     # a key block and one key
    (1, 4, 2, 333, 400, 64, 50, 9, False, BF16),
    (1, 3, 3, 640, 640, 128, 64, 256, False, BF16),
    (1, 2, 1, 1, 513, 128, 100, 5, True, BF16),
    (1, 1, 1, 9000, 9000, 64, 100, 2, True, BF16),      # the sinks' walk in many pieces
    (1, 2, 1, 300, 300, 64, 30, 500, True, BF16),       # more sinks than keys
])
def test_against_the_definition(swa, B, Hq, H, Lq, Lk, D, window, sinks, causal, dtype):
    g = torch.Generator(device="cuda").manual_seed(Lq + Lk + D)
    q, k = normal(g, B, Hq, Lq, D, dtype=dtype), normal(g, B, H, Lk, D, dtype=dtype)
    lse = lse_of(q, k, window, sinks, causal)
    want, tol = reference(q, k, lse, window, sinks, causal)
    got = torch.full((B, H, Lk), math.nan, device="cuda")
    need = swa.swa_attn_key_weights_workspace_bytes(B, Hq, H, Lq, Lk, D, window, causal, sinks)
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")
    swa.swa_attn_key_weights(q, k, lse, window, causal=causal, out=got, workspace=ws[:need] if need else None,
                             sinks=sinks)
    swa.swa_check_device()
    assert ((got.double() - want).abs() <= tol).all(), ((got.double() - want).abs() / tol).max()
    assert ((got.double().sum(-1) - Hq // H * Lq).abs() <= tol.sum(-1)).all()  # each row gives out one
    assert (ws[need:] == 255).all()
    assert torch.equal(swa.swa_attn_key_weights(q, k, lse, window, causal=causal, sinks=sinks), got)


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [(50, 0), (400, 7), (10**12, 7)])
def test_without_sinks_or_with_a_wide_window_nothing_changes(swa, window, sinks):
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k = normal(g, 1, 4, 400, 64), normal(g, 1, 2, 400, 64)
    lse = lse_of(q, k, window, sinks, True)
    assert torch.equal(swa.swa_attn_key_weights(q, k, lse, window, sinks=sinks),
                       swa.swa_attn_key_weights(q, k, lse, window))


@pytest.mark.gpu
def test_what_a_sink_does_not_see_stays_out(swa):
    """NaN in keys between the sinks and the windows, and in queries before a sink."""
    g = torch.Generator(device="cuda").manual_seed(2)
    q, k = normal(g, 1, 2, 600, 64), normal(g, 1, 1, 600, 64)
    lse = lse_of(q, k, 40, 300, True)
    clean = swa.swa_attn_key_weights(q, k, lse, 40, sinks=300)
    k2, q2 = k.clone(), q.clone()
    k2[:, :, 320:500] = math.nan
    q2[:, :, :250] = math.nan
    got = swa.swa_attn_key_weights(q2, k2, lse, 40, sinks=300)
    assert got[:, :, :250].isnan().all() and got[:, :, 320:500].isnan().all()
    for part in (slice(250, 320), slice(500, 600)):
        assert torch.equal(got[:, :, part], clean[:, :, part])


@pytest.mark.gpu
def test_a_prompt_and_its_steps_add_up(swa):
    """The weights of a prompt of N tokens, and those that the next tokens add over the cache, are the
    weights of the longer prompt; in a captured graph, with an eviction behind that keeps the heaviest."""
    H, Hq, D, W, S, N, T = 2, 4, 64, 96, 5, 500, 8
    g = torch.Generator(device="cuda").manual_seed(4)
    q = normal(g, 1, Hq, N + T, D)
    # keys and values that the cache holds exactly
    k, v = ((torch.randint(-8, 9, (1, H, N + T, D), generator=g, device="cuda") / 8).bfloat16()
            for _ in range(2))
    _, lse = swa.swa_attn_fwd(q, k, v, W, sinks=S)
    whole = swa.swa_attn_key_weights(q, k, lse, W, sinks=S)
    _, tol = reference(q, k, lse, W, S, True)
    cache = swa.SwaCache.empty(40, H, D, page=32)
    table = torch.arange(20, dtype=torch.int32, device="cuda")[None]
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    first = [t[:, :, :N].contiguous() for t in (q, k, v)]
    rest = [t[:, :, N:].contiguous() for t in (q, k, v)]

    def run():
        lens.zero_()
        _, z = swa.swa_attn_fwd(*first, W, sinks=S)
        w = swa.swa_attn_key_weights(first[0], first[1], z, W, sinks=S)
        swa.swa_cache_append(cache, table, lens, *first[1:], weight=w)
        lens.add_(N)
        swa.swa_cache_append(cache, table, lens, *rest[1:])
        swa.swa_cache_attn(rest[0], cache, table, lens, W, accumulate=True, sinks=S)
        lens.add_(T)

    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    cache.weight.zero_()
    graph.replay()
    torch.cuda.synchronize()
    got = cache.weight[:20].permute(1, 0, 2).reshape(1, H, -1)[:, :, :N + T].double()
    # both sides of the definition's tolerance, and the cached rows' lse: within 1e-3 of the forward's
    assert ((got - whole.double()).abs() <= 2 * tol + 2e-3 * whole.double()).all()
    swa.swa_check_device()
    kept, left = swa.swa_cache_evict(cache, table, lens, table + 20, budget=64, recent=16)
    assert left.item() == 64
    top = got[0, 0, :N + T - 16].topk(48).indices.sort().values
    assert torch.equal(kept[0, 0, :48].long(), top)


def test_refusals_and_sizes():
    import sliding_window_flash_gb300 as swa

    lib, fake = swa.load(), 1 << 20
    size = lib.swa_attn_key_weights_sinks_workspace_bytes

    def call(sinks=3, window=4, Lq=600, Lk=700, ws=fake, room=1 << 40, D=64, q=fake):
        return lib.swa_attn_key_weights_sinks(q, fake, fake, fake, 1, 4, 2, Lq, Lk, D, window, sinks, 1, 0.1, 0,
                                              ws, room, None)

    assert call(sinks=-1) == 1 and call(q=0) == 1 and call(window=0) == 1 and call(Lq=701) == 1
    assert call(D=96) == 2 and call(q=fake + 8) == 3 and call(ws=fake + 8) == 3
    plain = lib.swa_attn_key_weights_workspace_bytes
    assert size(1, 4, 2, 600, 700, 64, 4, 0, 1) == plain(1, 4, 2, 600, 700, 64, 4, 1)
    assert size(1, 4, 2, 600, 700, 64, 4, -1, 1) == 0 and size(1, 4, 2, 600, 700, 96, 4, 1, 1) == 0
    # wide windows hide nothing, and all keys are sinks at most
    assert size(1, 4, 2, 600, 700, 64, 700, 9, 1) == plain(1, 4, 2, 600, 700, 64, 700, 1)
    assert size(1, 4, 2, 600, 700, 64, 4, 10**9, 1) == size(1, 4, 2, 600, 700, 64, 4, 700, 1)
    need = size(1, 1, 1, 9000, 9000, 64, 4, 9000, 1)
    assert need > plain(1, 1, 1, 9000, 9000, 64, 4, 1)
    many = dict(sinks=700)
    assert call(**many, room=size(1, 4, 2, 600, 700, 64, 4, 700, 1) - 1) == 6 and call(**many, ws=0) == 6
