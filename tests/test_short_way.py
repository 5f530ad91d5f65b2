"""The binding's short way to the library (csrc/swa_torch.cpp) against the Python way, which does the same
calls: equal bits, the caller's tensors and workspaces used, the same refusals."""
import math

import pytest
import torch

import sliding_window_flash_gb300 as swa_pkg
from sliding_window_flash_gb300 import cache as mod

NONE = {n: (lambda *_: None) for n in ("attn", "fwd", "bwd")}


@pytest.fixture(params=["short", "python"])
def way(request, monkeypatch):
    """Both ways, and how many calls the short one answered."""
    mod._t.f32  # the names are loaded
    answered = []
    for n in NONE:
        fn = getattr(mod._t, n) if request.param == "short" else NONE[n]

        def call(*args, fn=fn):
            r = fn(*args)
            if r is not None:
                answered.append(r)
            return r

        monkeypatch.setitem(mod._t.__dict__, n, call)
    return request.param, answered


def test_it_is_built_and_leaves_what_is_no_cuda_tensor():
    mod._t.f32
    assert type(mod._t.attn).__name__ == "builtin_function_or_method"
    x = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16)
    assert mod._t.fwd(x, x, x, None, None, None, 4, None, True, 1) is None
    assert mod._t.bwd(*[x] * 5, None, None, None, None, None, 4, None, True, 1) is None
    held = (x, x, x, x, None, x.device, (1, 1, 1, 64))
    assert mod._t.attn(held, x, x, x, None, None, None, None, 4, None, False, 0, 0) is None
    assert mod._t.pool(x, x, x, x, None) is None and mod._t.pool(None) is None
    for bad in ((), (1,), (held,) * 13, (None,) * 13, (None,) * 10, (None,) * 14):
        for n in NONE:
            assert getattr(mod._t, n)(*bad) is None


def layer(dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn((2, 4, 200, 64), generator=g, device="cuda").to(dtype)
    k, v = (torch.randn((2, 2, 300, 64), generator=g, device="cuda").to(dtype) for _ in range(2))
    return q, k, v, torch.randn((2, 4, 200, 64), generator=g, device="cuda").to(dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("given", [False, True])
def test_layer(swa, way, dtype, given):
    name, answered = way
    q, k, v, do = layer(dtype)
    kw, kb = {}, {}
    if given:
        need = [max(16, swa.swa_attn_sinks_workspace_bytes(2, 4, 2, 200, 300, 64, 40, 3, dtype=dtype,
                                                           backward=b)) for b in (False, True)]
        kw = dict(out=torch.empty_like(q), lse=q.new_empty((2, 4, 200), dtype=torch.float32),
                  workspace=torch.empty(need[0], dtype=torch.uint8, device="cuda"))
        kb = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v),
                  workspace=torch.empty(need[1], dtype=torch.uint8, device="cuda"))
    o, lse = swa.swa_attn_fwd(q, k, v, 40, sinks=3, **kw)
    grads = swa.swa_attn_bwd(q, k, v, o, do, lse, 40, sinks=3, **kb)
    assert len(answered) == (2 if name == "short" else 0)
    if given:
        assert o is kw["out"] and lse is kw["lse"]
        assert all(a is b for a, b in zip(grads, (kb["dq"], kb["dk"], kb["dv"])))
    got = [t.clone() for t in (o, lse, *grads)]
    for n in NONE:
        mod._t.__dict__[n] = NONE[n]
    o, lse = swa.swa_attn_fwd(q, k, v, 40, 1 / math.sqrt(64), sinks=3)
    for a, b in zip(got, (o, lse, *swa.swa_attn_bwd(q, k, v, o, do, lse, 40, sinks=3))):
        assert a.dtype == b.dtype and torch.equal(a, b) and not a.requires_grad


def pool(weight=False, B=2, pages=5, page=32):
    g = torch.Generator(device="cuda").manual_seed(4)
    cache = swa_pkg.SwaCache.empty(B * pages, 2, 64, page, weight=weight)
    table = torch.arange(B * pages, device="cuda", dtype=torch.int32).reshape(B, pages)
    lens = torch.zeros(B, device="cuda", dtype=torch.int32)
    kv = [torch.randn((B, 2, 150, 64), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]
    swa_pkg.swa_cache_append(cache, table, lens, *kv)
    return cache, table, lens + 140, torch.randn((B, 4, 3, 64), generator=g, device="cuda").to(torch.bfloat16)


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [dict(), dict(sinks=2), dict(shared=2), dict(sinks=2, accumulate=True),
                                dict(new=True, sinks=1), dict(given=True, shared=1), dict(scale=0.25)],
                         ids=lambda kw: "_".join(kw) or "plain")
def test_cache(swa, way, kw):
    name, answered = way
    kw = dict(kw)
    cache, table, lens, q = pool(weight=kw.get("accumulate", False))
    if "shared" in kw:  # (never with accumulate: two sequences would add to the same weights)
        table[1, :2] = table[0, :2]
    given = kw.pop("given", False)
    if kw.pop("new", False):
        kw["new"] = torch.tensor([3, 1], device="cuda", dtype=torch.int32)
    outs = {}
    if given:
        need = swa.swa_cache_attn_workspace_bytes(2, 4, 2, 3, 64, 5, 32, window=50, shared=1)
        outs = dict(out=torch.empty_like(q), lse=torch.empty((2, 4, 3), device="cuda"),
                    workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
    before = cache.weight.clone() if cache.weight is not None else None
    o, lse = swa.swa_cache_attn(q, cache, table, lens, 50, **kw, **outs)
    assert len(answered) == (1 if name == "short" else 0)
    if given:
        assert o is outs["out"] and lse is outs["lse"]
    after = cache.weight.clone() if before is not None else None
    for n in NONE:
        mod._t.__dict__[n] = NONE[n]
    if before is not None:
        cache.weight.copy_(before)
    o2, lse2 = swa.swa_cache_attn(q, cache, table, lens, 50, **kw)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    if before is not None:
        assert torch.equal(after, cache.weight) and not torch.equal(after, before)


@pytest.mark.gpu
def test_ints_past_32_bits_and_other_numbers(swa, way):
    name, answered = way
    q, k, v, _ = layer()
    for window, sinks, scale in ((2**40, 3, None), (2**31 - 1, 2**40, 0.1), (40, 2**70, 1)):
        o, _ = swa.swa_attn_fwd(q, k, v, window, scale, sinks=sinks)
        w, _ = swa.swa_attn_fwd(q, k, v, 300, scale)
        assert torch.equal(o, w)
    assert len(answered) == (2 if name == "short" else 0)  # an int for a scale is Python's


@pytest.mark.gpu
def test_refusals_are_the_same(swa, way):
    q, k, v, do = layer()
    o, lse = swa.swa_attn_fwd(q, k, v, 40, sinks=3)
    cache, table, lens, q1 = pool()
    small = torch.empty(16, dtype=torch.uint8, device="cuda")

    def fwd(q=q, k=k, v=v, window=40, sinks=3, **kw):
        swa.swa_attn_fwd(q, k, v, window, sinks=sinks, **kw)

    def bwd(do=do, lse=lse, **kw):
        swa.swa_attn_bwd(q, k, v, o, do, lse, 40, sinks=3, **kw)

    def attn(q=q1, table=table, lens=lens, window=50, **kw):
        swa.swa_cache_attn(q, cache, table, lens, window, **kw)

    for call, error in (
            (lambda: fwd(k=k.half()), TypeError), (lambda: fwd(v=v[:, :, 1:]), ValueError),
            (lambda: fwd(q=q.cpu()), ValueError), (lambda: fwd(q=q.mT), ValueError),
            (lambda: fwd(q=q[0]), ValueError), (lambda: fwd(sinks=-1), ValueError),
            (lambda: fwd(window=0), swa.SwaError), (lambda: fwd(scale=-1.0), swa.SwaError),
            (lambda: fwd(scale=math.nan), swa.SwaError), (lambda: fwd(out=q.half()), TypeError),
            (lambda: fwd(lse=lse[:1]), ValueError), (lambda: fwd(workspace=small.cpu()), ValueError),
            (lambda: fwd(q=k, k=q[:, :, :150], v=q[:, :, :150]), ValueError),
            (lambda: bwd(do=do.float()), TypeError), (lambda: bwd(lse=lse.half()), TypeError),
            (lambda: bwd(workspace=small), swa.SwaError), (lambda: bwd(dk=q), ValueError),
            (lambda: bwd(workspace=torch.empty((64, 64), device="cuda")[:, 1:]), ValueError),
            (lambda: attn(q=q1.float()), TypeError), (lambda: attn(table=table.long()), TypeError),
            (lambda: attn(lens=lens[:1]), ValueError), (lambda: attn(window=0), swa.SwaError),
            (lambda: attn(sinks=-1), swa.SwaError), (lambda: attn(shared=6), swa.SwaError),
            (lambda: attn(shared=-1), swa.SwaError), (lambda: attn(workspace=small), swa.SwaError),
            (lambda: attn(accumulate=True), swa.SwaError), (lambda: attn(new=lens.long()), TypeError),
            (lambda: attn(out=q1[:, :, :2]), ValueError), (lambda: attn(scale=0.0), swa.SwaError)):
        with pytest.raises(error):
            call()
    swa.swa_check_device()


@pytest.mark.gpu
def test_on_a_side_stream_and_captured(swa):
    q, k, v, _ = layer()
    cache, table, lens, q1 = pool()
    want = [*swa.swa_attn_fwd(q, k, v, 40, sinks=3), *swa.swa_cache_attn(q1, cache, table, lens, 50, sinks=2)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = [*swa.swa_attn_fwd(q, k, v, 40, sinks=3), *swa.swa_cache_attn(q1, cache, table, lens, 50, sinks=2)]
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("weight", [False, True])
def test_pools(swa, weight, monkeypatch):
    a = swa.SwaCache.empty(3, 2, 64, 32, weight=weight)
    assert mod._t.pool(*a.held[:5]) == a.held
    monkeypatch.setitem(mod._t.__dict__, "pool", lambda *_: None)
    b = swa.SwaCache(*a.held[:5])
    assert [type(x) for x in a.held] == [type(x) for x in b.held]
    assert all(x is y for x, y in zip(a.held[:5], b.held[:5])) and a.held[5:] == b.held[5:]
    assert (a.page, a.shape, a.device) == (32, (3, 2, 32, 64), a.k.device) == (b.page, b.shape, b.device)


@pytest.mark.gpu
def test_pools_that_are_refused(swa):
    k, v, ks, vs, w = swa.SwaCache.empty(3, 2, 64, 32).held[:5]
    for args, error in (((k, v[:2], ks, vs), ValueError), ((k, v.view(torch.uint8), ks, vs), TypeError),
                        ((k, v, ks.double(), vs), TypeError), ((k, v, ks, vs[:, :1]), ValueError),
                        ((k, v, ks, vs, w[:, :, :16]), ValueError), ((k, v.cpu(), ks, vs), ValueError),
                        ((k[0], v, ks, vs), ValueError), ((k.mT, v.mT, ks, vs), ValueError),
                        ((k, v, None, vs), TypeError)):
        with pytest.raises(error):
            swa.SwaCache(*args)
