"""Cache attention with sinks on the GPU against its definition in 64 bits: query t of sequence b at slot
p = lens[b] + t sees slots s <= p with p - s < window or s < sinks."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16


def make(swa, seed, pages, H, D, page, spread=3, weight=True):
    """A pool full of codes whose block scales differ by up to 2^spread."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def codes():
        x = torch.randn((pages, H, page, D), generator=g, device="cuda") * 90
        return x.clamp(-448, 448).to(torch.float8_e4m3fn)

    def scales():
        return torch.exp2(torch.randint(-8, -7 + spread, (pages, H), generator=g, device="cuda").float())

    w = torch.exp(torch.randn((pages, H, page), generator=g, device="cuda")) if weight else None
    return swa.SwaCache(codes(), codes(), scales(), scales(), w), g


def ints(v):
    return None if v is None else torch.tensor(v, dtype=torch.int32, device="cuda")


def attn_ref(cache, table, lens, q, window, sinks, new=None):
    """(o, lse, added weights, their tolerances): the tolerances from the arithmetic that a kernel may use.  A
    score is an fp32 sum of D products, each step and the rounding of the scaled score 2^-24: es = (D + 8)
    2^-24 scale <|q|, |k|> plus 2^-21 for the exponential; p is rounded to fp16 (2^-11, or 2^-25 where it
    is subnormal); o is rounded once to its type; weights are added in fp32."""
    B, Hq, T, D = q.shape
    H, S = cache.k.shape[1], cache.page
    G = Hq // H
    f64 = dict(dtype=torch.float64, device="cuda")
    k, v = cache.k.float().double(), cache.v.float().double()
    ks, vs = cache.k_scale.double(), cache.v_scale.double()
    o, lse = torch.zeros((B, Hq, T, D), **f64), torch.full((B, Hq, T), -math.inf, **f64)
    to, tl = torch.zeros_like(o), torch.zeros_like(lse)
    add, ta = torch.zeros(cache.k.shape[:3], **f64), torch.zeros(cache.k.shape[:3], **f64)
    half = torch.finfo(q.dtype).eps / 2
    for b in range(B):
        for t in range(T if new is None else new[b]):
            p = lens[b] + t
            s = torch.arange(p + 1, device="cuda")
            s = s[(p - s < window) | (s < sinks)]
            page = table[b].long()[s // S]
            for h in range(H):
                kk = k[page, h, s % S] * ks[page, h, None]
                vv = v[page, h, s % S] * vs[page, h, None]
                qq = q[b, h * G:(h + 1) * G, t].double()
                x = qq @ kk.T / math.sqrt(D)
                es = ((D + 8) * 2.0**-24 / math.sqrt(D) * (qq.abs() @ kk.abs().T)).amax(-1, keepdim=True)
                es = es + 2.0**-21
                z = torch.logsumexp(x, -1, keepdim=True)
                e = torch.exp(x - z)
                r = e @ vv
                row = (b, slice(h * G, (h + 1) * G), t)
                o[row], lse[row] = r, z[:, 0]
                to[row] = (e @ vv.abs()) * (2.0**-11 + 2 * es) + 2.0**-25 * vv.abs().sum(0) + \
                    1.01 * half * r.abs() + (2.0**-25 if q.dtype == FP16 else 0.0)
                tl[row] = (es + 2.0**-22 * (1 + z.abs()))[:, 0]
                add[page, h, s % S] += e.sum(0)
                ta[page, h, s % S] += (e * (3 * es + 2.0**-21 * (x.abs() + 1))).sum(0)
    return o, lse, add, to, tl, ta


def near(got, want, tol, what):
    got = got.double()
    fine = torch.isfinite(want)
    assert torch.equal(got[~fine], want[~fine]), what
    off = (got - want)[fine].abs()
    assert (off <= tol[fine]).all(), (what, (off / tol[fine].clamp(min=1e-300)).max().item())


CASES = [
    # B, Hq, H, D, page, T, lens, window, sinks, new, dtype
    (1, 1, 1, 64, 32, 1, [0], 1, 1, None, BF16),
    (3, 2, 2, 128, 64, 1, [0, 1, 700], 1, 1, None, BF16),
    (4, 4, 2, 128, 64, 1, [40, 64, 500, 901], 64, 4, None, BF16),
    (3, 4, 2, 128, 32, 3, [31, 500, 77], 33, 32, [3, 0, 2], BF16),
    (3, 8, 1, 64, 64, 5, [300, 0, 900], 100, 33, None, FP16),
    (2, 6, 2, 256, 32, 2, [700, 45], 50, 17, None, FP16),
    (2, 7, 1, 128, 128, 8, [333, 900], 129, 300, [8, 5], BF16),
    (2, 16, 1, 128, 64, 7, [1000, 130], 200, 4, None, BF16),     # two tiles of rows
    (3, 2, 1, 256, 128, 1, [1000, 200, 1], 7, 900, None, BF16),  # more sinks than some have tokens
    (2, 2, 2, 64, 64, 64, [500, 0], 32, 65, [64, 33], FP16),
    (70, 4, 1, 64, 32, 1, list(range(0, 1400, 20)), 30, 5, None, BF16),
]


@pytest.mark.parametrize("acc", [False, True], ids=["", "weights"])
@pytest.mark.parametrize("B,Hq,H,D,page,T,lens,window,sinks,new,dtype", CASES)
def test_attn(swa, B, Hq, H, D, page, T, lens, window, sinks, new, dtype, acc):
    width = -(-(max(lens) + T) // page)
    cache, g = make(swa, B * 100 + T, B * width + 1, H, D, page)
    table = torch.randperm(B * width, generator=g, device="cuda").to(torch.int32).view(B, width)
    q = torch.randn((B, Hq, T, D), generator=g, device="cuda").to(dtype)
    o, lse, add, to, tl, ta = attn_ref(cache, table, lens, q, window, sinks, new)
    before = cache.weight.double()
    got_o, got_lse = swa.swa_cache_attn(q, cache, table, ints(lens), window, new=ints(new), sinks=sinks,
                                        accumulate=acc)
    swa.swa_check_device()
    near(got_o, o, to, "o")
    near(got_lse, lse, tl, "lse")
    if acc:
        near(cache.weight, before + add, ta + 2.0**-23 * (before + add), "weights")
        assert torch.equal(cache.weight[add == 0], before[add == 0].float())
    else:
        assert torch.equal(cache.weight.double(), before)


def test_no_sinks_and_wide_windows_change_nothing(swa):
    cache, g = make(swa, 1, 40, 2, 128, 64)
    table = torch.arange(40, dtype=torch.int32, device="cuda").view(2, 20)
    q, lens = torch.randn((2, 4, 2, 128), generator=g, device="cuda").bfloat16(), ints([1000, 300])
    for window, sinks, like in ((100, 0, 100), (1280, 9, 1280), (2**40, 9, 1280), (200, 2**40, 1280)):
        a = swa.swa_cache_attn(q, cache, table, lens, window, sinks=sinks)
        b = swa.swa_cache_attn(q, cache, table, lens, like)
        swa.swa_check_device()
        for x, y in zip(a, b):
            assert torch.equal(x, y) or sinks == 2**40
            assert (x.double() - y.double()).norm() <= 2.0**-8 * y.double().norm()


def test_pages_between_are_not_read(swa):
    """Table entries between the sinks and the windows may name no page; NaN beside the sinks, and beside
    the window, reaches nobody."""
    cache, g = make(swa, 2, 40, 2, 64, 32)
    table = torch.arange(40, dtype=torch.int32, device="cuda").view(2, 20).contiguous()
    q, lens = torch.randn((2, 4, 1, 64), generator=g, device="cuda").bfloat16(), ints([600, 500])
    clean = swa.swa_cache_attn(q, cache, table, lens, 40, sinks=5)
    holed = table.clone()
    holed[:, 1:14] = -7
    nan = torch.tensor(0x7F, dtype=torch.uint8, device="cuda")
    for t in (cache.k, cache.v):
        t.view(torch.uint8)[::20, :, 5:] = nan          # the sinks' own pages
        t.view(torch.uint8)[17, :, :17] = nan           # slots 544 .. 560 of sequence 0, window from 561
    got = swa.swa_cache_attn(q, cache, holed, lens, 40, sinks=5)
    swa.swa_check_device()
    for a, b in zip(got, clean):
        assert torch.equal(a, b)


def test_a_bad_page_of_sinks_is_skipped_and_reported(swa):
    cache, g = make(swa, 3, 40, 1, 128, 64)
    table = torch.arange(40, dtype=torch.int32, device="cuda").view(2, 20).contiguous()
    q = torch.randn((2, 2, 1, 128), generator=g, device="cuda").bfloat16()
    bad = table.clone()
    bad[1, 0] = 40
    got = swa.swa_cache_attn(q, cache, bad, ints([1000, 1000]), 70, sinks=9)
    with pytest.raises(swa.SwaError, match="INDEX"):
        swa.swa_check_device()
    want = swa.swa_cache_attn(q, cache, table, ints([1000, 1000]), 70, sinks=9)
    plain = swa.swa_cache_attn(q, cache, table, ints([1000, 1000]), 70)
    swa.swa_check_device()
    for a, b, c in zip(got, want, plain):
        assert torch.equal(a[0], b[0])
        assert (a[1].double() - c[1].double()).norm() <= 2.0**-8 * c[1].double().norm()


def test_a_step_of_training_and_serving_together(swa):
    """A prompt through the training forward with sinks, its keys into the cache, then single tokens in a
    captured graph: each answers as the training forward does for the longer sequence."""
    H, Hq, D, W, S, N, steps = 2, 4, 64, 96, 5, 500, 6
    g = torch.Generator(device="cuda").manual_seed(4)
    q = torch.randn((1, Hq, N + steps, D), generator=g, device="cuda").bfloat16()
    # values that the cache holds exactly
    k, v = ((torch.randint(-8, 9, (1, H, N + steps, D), generator=g, device="cuda") / 8).bfloat16()
            for _ in range(2))
    cache = swa.SwaCache.empty(20, H, D, page=32, weight=False)
    table, lens = torch.arange(20, dtype=torch.int32, device="cuda")[None], ints([0])
    swa.swa_cache_append(cache, table, lens, k[:, :, :N].contiguous(), v[:, :, :N].contiguous())
    lens += N
    want, want_lse = swa.swa_attn_fwd(q, k, v, W, sinks=S)
    q1, k1, v1 = (t[:, :, N:N + 1].contiguous() for t in (q, k, v))
    swa.swa_cache_attn(q1, cache, table, lens, W, sinks=S)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        swa.swa_cache_append(cache, table, lens, k1, v1)
        o, lse = swa.swa_cache_attn(q1, cache, table, lens, W, sinks=S)
        lens += 1
    for t in range(N, N + steps):
        for dst, src in ((q1, q), (k1, k), (v1, v)):
            dst.copy_(src[:, :, t:t + 1])
        graph.replay()
        torch.cuda.synchronize()
        ref = want[:, :, t:t + 1].double()
        # both forms round P (2^-9 in bf16, 2^-11) and o (2^-9 each)
        assert (o.double() - ref).norm() <= 1e-2 * ref.norm()
        assert (lse - want_lse[:, :, t:t + 1]).abs().max() <= 1e-3
    swa.swa_check_device()
