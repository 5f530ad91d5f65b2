"""Calls whose kernels may be launched before the work ahead of them in the stream has ended: what comes
before (kernels, copies, fills, other streams, other calls) is waited for, eager and captured, and what comes
behind sees everything.  Each run is compared, bit for bit, with one that waits for the GPU between all steps."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
D64, D128, D256 = (1, 4, 2, 300, 64), (1, 3, 1, 300, 128), (1, 2, 1, 300, 256)


def normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").to(BF16)


def training(swa, sizes, settle):
    """Layers whose inputs are written by kernels, copies and fills directly ahead, and changed behind."""
    B, Hq, H, N, D = sizes
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = normal(g, B, H, N, D), normal(g, B, H, N, D)
    source, q, do = normal(g, B, Hq, N, D), torch.empty((B, Hq, N, D), dtype=BF16, device="cuda"), None
    big = torch.randn((1024, 1024), generator=g, device="cuda")

    def run():
        total = torch.zeros_like(source)
        for i in range(4):
            busy = big @ big @ big  # keeps the GPU at work ahead of the copy
            settle()
            q.copy_(source)
            settle()
            o, lse = swa.swa_attn_fwd(q, k, v, 40, sinks=3 + i)
            settle()
            q.zero_()  # after the forward has read it
            settle()
            q.copy_(source)
            settle()
            dq, dk, dv = swa.swa_attn_bwd(q, k, v, o, o, lse, 40, sinks=3 + i)
            settle()
            total.add_(dq).add_(o)
            k.add_(dk, alpha=2.0**-6)
            v.sub_(dv, alpha=2.0**-6)
            settle()
        return total, k, v, busy

    return run


def serving(swa, sizes, settle):
    """Steps of append, attention (three forms) and eviction, each on what the one ahead has written."""
    B, Hq, H, N, D = 3, *sizes[1:]
    g = torch.Generator(device="cuda").manual_seed(2)
    cache = swa.SwaCache.empty(120, H, D, page=32)
    for t in (cache.k, cache.v, cache.weight):
        t.view(torch.uint8).zero_()
    table = torch.arange(60, dtype=torch.int32, device="cuda").reshape(B, 20).contiguous()
    table[:, :2] = table[0, :2]
    spare = torch.arange(60, 120, dtype=torch.int32, device="cuda").reshape(B, 20).contiguous()
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    k0 = normal(g, 1, H, 64, D).expand(B, H, 64, D).contiguous()
    ks = [normal(g, B, H, 70, D) for _ in range(3)]
    qs = [normal(g, B, Hq, 5, D) for _ in range(3)]
    buf = torch.empty_like(qs[0])

    def run():
        lens.zero_()
        cache.weight.zero_()
        swa.swa_cache_append(cache, table[:1], lens[:1], k0[:1], k0[:1])  # the shared pages, once
        lens.add_(64)
        settle()
        out = []
        for k, q in zip(ks, qs):
            swa.swa_cache_append(cache, table, lens, k, k)
            settle()
            lens.add_(65)
            buf.copy_(q)
            settle()
            # (not the sinks: they lie on the shared pages, whose weights several sequences would add to)
            out += swa.swa_cache_attn(buf, cache, table, lens, 50, accumulate=True)
            settle()
            buf.neg_()
            settle()
            out += swa.swa_cache_attn(buf, cache, table, lens, 1000, sinks=2, shared=2)
            settle()
            out += swa.swa_cache_attn(buf, cache, table, lens, 30, sinks=3)
            settle()
            lens.add_(5)
        kept, left = swa.swa_cache_evict(cache, table, lens, spare, budget=100, recent=20)
        settle()
        out += swa.swa_cache_attn(buf, cache, spare, left - 5, 1000, sinks=1)
        return out + [kept, cache.weight]

    return run


@pytest.mark.parametrize("sizes", [D64, D128, D256], ids=["d64", "d128", "d256"])
@pytest.mark.parametrize("make", [training, serving])
def test_nothing_overtakes(swa, make, sizes):
    want = [t.clone() for t in make(swa, sizes, torch.cuda.synchronize)()]
    torch.cuda.synchronize()

    def same(got, how):
        torch.cuda.synchronize()
        swa.swa_check_device()
        for i, (a, b) in enumerate(zip(want, got)):
            assert torch.equal(a, b), f"{how}: output {i}"

    same(make(swa, sizes, lambda: None)(), "eager")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = make(swa, sizes, lambda: None)()
    torch.cuda.current_stream().wait_stream(side)
    same(got, "another stream")
    run = make(swa, sizes, lambda: None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    graph.replay()
    same(got, "captured")


@pytest.mark.parametrize("captured", [False, True])
def test_inputs_of_another_stream(swa, captured):
    """The call's stream waits for an event of a stream that is still at work on q, and that stream then for
    the call before it overwrites q."""
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v, first, second = (normal(g, 1, H, 500, 64) for H in (2, 2, 4, 4))
    big, q = torch.randn((2048, 2048), generator=g, device="cuda"), torch.zeros_like(first)
    wants = [swa.swa_attn_fwd(x, k, v, 40, sinks=3) for x in (first, second)]
    other = torch.cuda.Stream()

    def run():
        here, got = torch.cuda.current_stream(), []
        for x in (first, second):
            other.wait_stream(here)
            with torch.cuda.stream(other):
                big @ big @ big
                q.copy_(x)
            here.wait_stream(other)
            got.append(swa.swa_attn_fwd(q, k, v, 40, sinks=3))
            other.wait_stream(here)
            with torch.cuda.stream(other):
                q.zero_()
            here.wait_stream(other)
        return got

    torch.cuda.synchronize()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = run()
        graph.replay()
    else:
        got = run()
    torch.cuda.synchronize()
    for a, b in zip(wants, got):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("sizes", [D64, D128, D256], ids=["d64", "d128", "d256"])
def test_two_streams_at_once(swa, sizes):
    """Layers on one stream and serving steps on another, at the same time and time and again."""
    makes = (training, serving)
    wants = [[t.clone() for t in make(swa, sizes, torch.cuda.synchronize)()] for make in makes]
    streams = [torch.cuda.Stream() for _ in makes]
    torch.cuda.synchronize()
    gots = [[], []]
    for _ in range(6):
        for make, stream, got in zip(makes, streams, gots):
            with torch.cuda.stream(stream):
                got.append(make(swa, sizes, lambda: None)())
    torch.cuda.synchronize()
    swa.swa_check_device()
    for want, runs in zip(wants, gots):
        for got in runs:
            for i, (a, b) in enumerate(zip(want, got)):
                assert torch.equal(a, b), i
