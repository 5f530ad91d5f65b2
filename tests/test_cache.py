"""The paged 8-bit cache on the GPU against plain 64-bit forms (cache_ref.py): append, attention,
eviction, key weights, and a run of them together."""
import math

import pytest
import torch

import cache_ref as ref

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _cache(swa, g, pages, H, D, page, spread=0, weight=True):
    """A pool full of codes; block scales differ by up to 2^spread."""
    def codes():
        x = torch.randn((pages, H, page, D), generator=g, device="cuda") * 90
        return x.clamp(-448, 448).to(torch.float8_e4m3fn)

    def scales():
        e = torch.randint(-8, -7 + spread, (pages, H), generator=g, device="cuda")
        return torch.exp2(e.float())

    w = torch.exp(torch.randn((pages, H, page), generator=g, device="cuda")) if weight else None
    return swa.SwaCache(codes(), codes(), scales(), scales(), w)


def _table(g, B, width, first=0):
    order = torch.randperm(B * width, generator=g, device="cuda") + first
    return order.to(torch.int32).view(B, width).contiguous()


def _ints(v):
    return None if v is None else torch.tensor(v, dtype=torch.int32, device="cuda")


def _same_pool(cache, want):
    got = ref.pool_of(cache)
    for name, x in want.items():
        if x is not None:
            assert torch.equal(torch.nan_to_num(got[name], nan=1e9),
                               torch.nan_to_num(x, nan=1e9)), name


def _near(got, want, tol, what):
    got = got.cpu().double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    fine = torch.isfinite(want)
    assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)]), what
    off = (got - want)[fine].abs()
    assert (off <= tol[fine]).all(), (what, float((off - tol[fine]).max()),
                                     float((off / tol[fine].clamp(min=1e-300)).max()))


# ---- append ------------------------------------------------------------------------------------

@pytest.mark.parametrize("B,H,D,page,T,lens,new,dtype,given", [
    (1, 1, 64, 32, 1, [0], None, torch.bfloat16, False),
    (3, 2, 128, 64, 1, [0, 63, 64], None, torch.bfloat16, False),
    (4, 2, 128, 64, 1, [1, 62, 127, 5], None, torch.float16, True),
    (2, 3, 128, 64, 200, [0, 37], None, torch.bfloat16, True),
    (3, 1, 256, 32, 45, [31, 0, 33], [45, 0, 17], torch.float16, False),
    (2, 2, 64, 128, 129, [127, 1], [129, 1], torch.float32, True),
    (1, 2, 256, 128, 300, [5], None, torch.float32, False),
    (2, 1, 128, 32, 33, [0, 31], [33, 32], torch.bfloat16, True),
])
def test_append(swa, B, H, D, page, T, lens, new, dtype, given):
    g = _gen(B * 1000 + T)
    width = -(-(max(lens) + T) // page)
    cache = _cache(swa, g, B * width + 2, H, D, page, spread=3)
    table = _table(g, B, width, first=1)
    pool = ref.pool_of(cache)
    # token magnitudes from 2^-6 to 2^6 raise some scales and leave others
    mag = torch.exp2(torch.randint(-6, 7, (B, H, T, 1), generator=g, device="cuda").float())
    k = (torch.randn((B, H, T, D), generator=g, device="cuda") * mag).to(dtype)
    v = (torch.randn((B, H, T, D), generator=g, device="cuda") * mag.flip(2)).to(dtype)
    w = torch.rand((B, H, T), generator=g, device="cuda") if given else None
    ref.append(pool, table, lens, k, v, new, w)
    for _ in range(2):  # again: the same slots, the same codes
        swa.swa_cache_append(cache, table, _ints(lens), k, v, new=_ints(new), weight=w)
        swa.swa_check_device()
        _same_pool(cache, pool)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_append_extreme_values(swa, dtype):
    """Zeros, values at and above the ends of the scales' range, the borders between two scales,
    and tokens that are not finite."""
    g = _gen(5)
    T, D, page = 96, 64, 32
    cache = _cache(swa, g, 4, 1, D, page)
    table = _table(g, 1, 4)
    k = torch.randn((1, 1, T, D), generator=g, device="cuda")
    v = torch.randn((1, 1, T, D), generator=g, device="cuda")
    k[0, 0, :32] = 0.0
    v[0, 0, :32] = 448.0 * 2.0**-30
    v[0, 0, 3, 1] = -448.0 * 2.0**-30
    k[0, 0, 40, 3] = math.nan
    v[0, 0, 41, 5] = math.inf
    k[0, 0, 42, 0] = -math.inf
    v[0, 0, 43, 63] = 1e30
    k[0, 0, 64:] *= 2.0**-60
    v[0, 0, 70, 7] = 448.0 * 2.0**40
    if dtype == torch.float32:
        k[0, 0, 32, 0] = 448.00003
    k, v = k.to(dtype), v.to(dtype)
    pool = ref.pool_of(cache)
    ref.append(pool, table, [0], k, v)
    swa.swa_cache_append(cache, table, _ints([0]), k, v)
    swa.swa_check_device()
    _same_pool(cache, pool)
    assert float(pool["k_scale"][int(table[0, 0]), 0]) == 2.0**-48
    assert torch.isnan(pool["k"][int(table[0, 1]), 0, 8:12]).all()


def test_append_without_weights_and_untouched_rows(swa):
    g = _gen(6)
    cache = _cache(swa, g, 5, 2, 128, 64, weight=False)
    before = cache.k.view(torch.uint8).clone()
    table = _ints([[3, 1], [0, 4]])
    k = torch.randn((2, 2, 3, 128), generator=g, device="cuda").bfloat16()
    swa.swa_cache_append(cache, table, _ints([62, 0]), k, k, new=_ints([3, 0]))
    swa.swa_check_device()
    now = cache.k.view(torch.uint8)
    for p in (0, 2, 4):
        assert torch.equal(now[p], before[p])
    assert torch.equal(now[1, :, 1:], before[1, :, 1:])
    assert not torch.equal(now[3, :, 62:], before[3, :, 62:])


# ---- attention ---------------------------------------------------------------------------------

ATTN = [
    # B, Hq, H, D, page, T, lens, window, new, dtype, accumulate
    (1, 1, 1, 64, 32, 1, [0], 1, None, torch.bfloat16, True),
    (2, 2, 2, 128, 64, 1, [0, 1], 1000, None, torch.bfloat16, True),
    (3, 4, 2, 128, 64, 1, [63, 64, 65], 1000, None, torch.bfloat16, True),
    (3, 4, 2, 128, 64, 1, [700, 300, 5], 100, None, torch.float16, True),
    (2, 8, 1, 64, 32, 1, [511, 1000], 64, None, torch.bfloat16, False),
    (2, 6, 2, 256, 128, 1, [400, 129], 5000, None, torch.float16, True),
    (1, 16, 1, 128, 64, 1, [2500], 5000, None, torch.bfloat16, True),
    (1, 40, 2, 128, 64, 1, [777], 5000, None, torch.bfloat16, True),
    (2, 4, 2, 128, 64, 5, [200, 60], 1000, None, torch.bfloat16, True),
    (3, 4, 2, 128, 32, 7, [200, 60, 0], 33, [7, 0, 3], torch.float16, True),
    (2, 14, 2, 64, 64, 4, [90, 350], 128, [1, 4], torch.bfloat16, True),
    (1, 4, 2, 256, 64, 3, [1000], 64, None, torch.bfloat16, True),
    (1, 4, 1, 128, 64, 64, [300], 5000, None, torch.bfloat16, True),
    (1, 4, 2, 256, 32, 33, [100], 40, None, torch.float16, True),
    (2, 2, 2, 64, 128, 16, [0, 5], 1, None, torch.bfloat16, True),
    (5, 4, 4, 128, 64, 1, [0, 31, 4000, 32, 95], 10000, None, torch.bfloat16, True),
    (40, 2, 1, 64, 32, 1, [3 * i for i in range(40)], 50, None, torch.float16, True),
    (1, 2, 1, 128, 64, 1, [20000], 30000, None, torch.bfloat16, True),
    # so many rows that a warp joins each
    (4, 64, 16, 128, 64, 4, [900, 350, 0, 620], 2000, None, torch.bfloat16, True),
    (4, 32, 16, 256, 128, 5, [300, 350, 128, 620], 200, [5, 0, 3, 1], torch.float16, True),
    (9, 40, 20, 64, 32, 2, [100 + 61 * i for i in range(9)], 500, None, torch.bfloat16, True),
    (8, 64, 16, 64, 32, 2, [100 + 97 * i for i in range(8)], 300, None, torch.float16, True),
    (8, 32, 16, 256, 64, 4, [90 + 53 * i for i in range(8)], 200, None, torch.bfloat16, False),
    # a warp joins 16 columns of a row
    (6, 16, 4, 128, 64, 2, [700, 0, 31, 1200, 64, 333], 800, [2, 1, 0, 2, 1, 2], torch.bfloat16, True),
]


@pytest.mark.parametrize("B,H_q,H,D,page,T,lens,window,new,dtype,acc", ATTN)
def test_attn(swa, B, H_q, H, D, page, T, lens, window, new, dtype, acc):
    g = _gen(B + T + D + lens[0])
    width = -(-(max(lens) + T) // page) + 1
    cache = _cache(swa, g, B * width + 1, H, D, page, spread=6)
    table = _table(g, B, width)
    # rows behind a sequence's last token hold NaN codes
    for b in range(B):
        end = lens[b] + (T if new is None else new[b])
        for blk in range(end // page, width):
            row = max(0, end - blk * page)
            for x in (cache.k, cache.v):
                x.view(torch.uint8)[int(table[b, blk]), :, row:] = ref.E4M3_NAN
    q = torch.randn((B, H_q, T, D), generator=g, device="cuda").to(dtype)
    pool = ref.pool_of(cache)
    o, lse, to, tl, tw = ref.attn(pool, table, lens, q, window, new=new, accumulate=acc)
    go, gl = swa.swa_cache_attn(q, cache, table, _ints(lens), window, new=_ints(new),
                                accumulate=acc)
    swa.swa_check_device()
    _near(go, o, to, "o")
    _near(gl, lse, tl, "lse")
    if acc:
        _near(cache.weight, pool["weight"], tw, "weight")
    # the same bits again, and without touching the weights
    w = cache.weight.clone()
    go2, gl2 = swa.swa_cache_attn(q, cache, table, _ints(lens), window, new=_ints(new))
    assert torch.equal(go, go2) and torch.equal(gl, gl2) and torch.equal(w, cache.weight)


@pytest.mark.parametrize("B,H_q,H,D,page,T,lens,window,new,dtype,acc,longest", [
    (2, 8, 1, 128, 64, 5, [2000, 65], 1 << 20, None, torch.bfloat16, True, 700000),
    (3, 14, 2, 128, 32, 3, [900, 0, 33], 1 << 20, [3, 0, 2], torch.float16, True, 300000),
    (2, 24, 3, 64, 128, 3, [1500, 127], 1 << 20, None, torch.bfloat16, True, 250000),
    (2, 7, 1, 64, 64, 9, [31, 1100], 400000, [9, 4], torch.float16, False, 500000),
    (1, 8, 4, 64, 32, 64, [300], 1 << 20, None, torch.bfloat16, True, 200000),
    (40, 112, 16, 64, 32, 5, [1300, 1024] + [11 * b for b in range(38)], 1000, None, torch.float16,
     False, 1536),
    (40, 42, 14, 128, 32, 12, [1400, 90] + [7 * b for b in range(38)], 1200,
     [12 - b % 4 for b in range(40)], torch.bfloat16, True, 1536),
])
def test_attn_long_tables(swa, B, H_q, H, D, page, T, lens, window, new, dtype, acc, longest):
    """Many rows under a table (and window) for long sequences, whatever their lengths are: a warp has two
    tiles of rows.  What the table holds behind the last token is no page."""
    g = _gen(D + B)
    width = -(-(max(lens) + T) // page)
    cache = _cache(swa, g, B * width, H, D, page, spread=4)
    table = torch.full((B, longest // page), -1, dtype=torch.int32, device="cuda")
    table[:, :width] = _table(g, B, width)
    for b in range(B):
        table[b, -(-(lens[b] + (T if new is None else new[b])) // page):] = -1
    q = torch.randn((B, H_q, T, D), generator=g, device="cuda").to(dtype)
    pool = ref.pool_of(cache)
    o, lse, to, tl, tw = ref.attn(pool, table, lens, q, window, new=new, accumulate=acc)
    go, gl = swa.swa_cache_attn(q, cache, table, _ints(lens), window, new=_ints(new),
                                accumulate=acc)
    swa.swa_check_device()
    _near(go, o, to, "o")
    _near(gl, lse, tl, "lse")
    if acc:
        _near(cache.weight, pool["weight"], tw, "weight")
    again = swa.swa_cache_attn(q, cache, table, _ints(lens), window, new=_ints(new))
    assert torch.equal(go, again[0]) and torch.equal(gl, again[1])


def test_attn_reads_nothing_outside_the_window(swa):
    """Table entries of pages wholly before the window, or behind the last token, may name no page
    at all, and NaN tokens outside a query's range change nothing for it."""
    g = _gen(11)
    cache = _cache(swa, g, 12, 2, 128, 32)
    table = _table(g, 1, 12)
    lens, window, T = [200], 64, 2
    q = torch.randn((1, 4, T, 128), generator=g, device="cuda").bfloat16()
    pool = ref.pool_of(cache)
    o, lse, to, tl, _ = ref.attn(pool, table, lens, q, window)
    # slots 137..201 are seen; slot 136 shares page 4 with them
    bad = table.clone()
    bad[0, :4] = -1
    bad[0, 7:] = 1 << 30
    cache.k.view(torch.uint8)[int(table[0, 4]), :, :9] = ref.E4M3_NAN
    cache.v.view(torch.uint8)[int(table[0, 4]), :, :9] = ref.E4M3_NAN
    go, gl = swa.swa_cache_attn(q, cache, bad, _ints(lens), window)
    swa.swa_check_device()
    _near(go, o, to, "o")
    _near(gl, lse, tl, "lse")


def test_attn_nan_token_reaches_only_who_sees_it(swa):
    g = _gen(12)
    D, page, T = 64, 32, 4
    cache = swa.SwaCache.empty(4, 1, D, page)
    table = _table(g, 1, 4)
    k = torch.randn((1, 1, 60, D), generator=g, device="cuda").bfloat16()
    v = torch.randn((1, 1, 60, D), generator=g, device="cuda").bfloat16()
    k2, v2 = k.clone(), v.clone()
    v2[0, 0, 58, 3] = math.inf  # the third of the four new tokens
    q = torch.randn((1, 2, T, D), generator=g, device="cuda").bfloat16()
    swa.swa_cache_append(cache, table, _ints([0]), k, v)
    clean, _ = swa.swa_cache_attn(q, cache, table, _ints([56]), 1000)
    swa.swa_cache_append(cache, table, _ints([0]), k2, v2)
    o, lse = swa.swa_cache_attn(q, cache, table, _ints([56]), 1000, accumulate=True)
    swa.swa_check_device()
    assert torch.isfinite(o[:, :, :2].float()).all() and torch.isfinite(lse[:, :, :2]).all()
    assert torch.isnan(o[:, :, 2:].float()).all() and torch.isnan(lse[:, :, 2:]).all()
    _near(o[:, :, :2], clean[:, :, :2].cpu().double(),
          2.0**-3 * torch.ones((1, 2, 2, D), dtype=torch.float64), "rows before")


def test_attn_large_and_small_queries(swa):
    """Rows of very large and very small queries, and scores far apart."""
    g = _gen(13)
    cache = _cache(swa, g, 8, 1, 128, 64)
    table = _table(g, 1, 8)
    q = torch.randn((1, 4, 1, 128), generator=g, device="cuda")
    q[0, 0] *= 1e6
    q[0, 1] *= 1e-30
    q[0, 2] = 0
    q[0, 3, 0, 1:] *= 1e-6
    q = q.bfloat16()
    lens = [300]
    pool = ref.pool_of(cache)
    o, lse, to, tl, _ = ref.attn(pool, table, lens, q, 1000)
    go, gl = swa.swa_cache_attn(q, cache, table, _ints(lens), 1000)
    swa.swa_check_device()
    _near(go, o, to, "o")
    _near(gl, lse, tl, "lse")


def test_attn_bad_pages_and_lengths(swa):
    """What the device finds out of range is skipped and reported; other sequences are unharmed."""
    g = _gen(14)
    cache = _cache(swa, g, 9, 2, 64, 32)
    table = _table(g, 3, 3)
    q = torch.randn((3, 2, 1, 64), generator=g, device="cuda").bfloat16()
    good, _ = swa.swa_cache_attn(q, cache, table, _ints([40, 50, 60]), 1000)
    swa.swa_check_device()
    for lens, page in (([40, -1, 60], None), ([40, 96, 60], None), ([40, 50, 60], -7),
                       ([40, 50, 60], 9), ([40, 2**31 - 1, 60], None)):
        t = table.clone()
        if page is not None:
            t[1, 0] = page
        before = cache.weight.clone()
        o, lse = swa.swa_cache_attn(q, cache, t, _ints(lens), 1000, accumulate=True)
        with pytest.raises(swa.SwaError, match="INDEX"):
            swa.swa_check_device()
        swa.swa_check_device()
        assert torch.equal(o[0], good[0]) and torch.equal(o[2], good[2])
        if page is None:
            assert (o[1] == 0).all() and torch.isinf(lse[1]).all()
        else:
            assert torch.isfinite(o[1].float()).all()
        cache.weight.copy_(before)
    k = torch.randn((3, 2, 1, 64), generator=g, device="cuda").bfloat16()
    before = cache.k.view(torch.uint8).clone()
    t = table.clone()
    t[:, 1] = -1
    swa.swa_cache_append(cache, t, _ints([40, 96, -3]), k, k)
    with pytest.raises(swa.SwaError, match="INDEX"):
        swa.swa_check_device()
    assert torch.equal(before, cache.k.view(torch.uint8))


# ---- eviction ----------------------------------------------------------------------------------

@pytest.mark.parametrize("B,H,D,page,lens,budget,recent,ties", [
    (1, 1, 64, 32, [50], 20, 5, False),
    (2, 2, 128, 64, [300, 64], 64, 10, False),
    (3, 2, 128, 64, [64, 65, 0], 64, 64, False),
    (2, 1, 64, 32, [200, 33], 40, 0, True),
    (2, 3, 256, 32, [100, 500], 97, 13, True),
    (1, 2, 64, 128, [3000], 1000, 100, True),
    (1, 1, 64, 64, [9000], 1, 0, False),
    (1, 1, 64, 64, [1025], 1024, 1, True),
    (4, 2, 128, 64, [10, 20, 30, 40], 128, 4, False),
])
def test_evict(swa, B, H, D, page, lens, budget, recent, ties):
    g = _gen(sum(lens) + budget)
    width = -(-max(lens + [1]) // page)
    room = -(-budget // page)
    cache = _cache(swa, g, B * (width + room), H, D, page, spread=12)
    if ties:
        cache.weight.copy_(torch.round(cache.weight * 2) / 2)
    cache.weight[::3, :, 7] = math.nan
    cache.weight[1::3, :, 9] = -0.0
    cache.k.view(torch.uint8)[0, 0, 3] = ref.E4M3_NAN
    order = _table(g, B, width + room)
    table, dst = order[:, :width].contiguous(), order[:, width:].contiguous()
    pool = ref.pool_of(cache)
    kept, out = ref.evict(pool, table, lens, dst, budget, recent)
    gk, go = swa.swa_cache_evict(cache, table, _ints(lens), dst, budget, recent)
    swa.swa_check_device()
    assert torch.equal(go.cpu(), out)
    assert torch.equal(gk.cpu(), kept)
    _same_pool(cache, pool)


def test_evict_bad_pages_and_lengths(swa):
    g = _gen(21)
    cache = _cache(swa, g, 12, 1, 64, 32)
    order = _table(g, 3, 4)
    table, dst = order[:, :2].contiguous(), order[:, 2:].contiguous()
    good = swa.swa_cache_evict(cache, table, _ints([64, 50, 40]), dst, 33, 4)[0].clone()
    swa.swa_check_device()
    for lens, where, value in (([64, -1, 40], None, 0), ([64, 65, 40], None, 0),
                               ([64, 50, 40], "table", 12), ([64, 50, 40], "dst", -1)):
        t, d = table.clone(), dst.clone()
        if where:
            (t if where == "table" else d)[1, 0] = value
        kept, out = swa.swa_cache_evict(cache, t, _ints(lens), d, 33, 4)
        with pytest.raises(swa.SwaError, match="INDEX"):
            swa.swa_check_device()
        assert torch.equal(kept[0], good[0]) and torch.equal(kept[2], good[2])
        if where is None:
            assert int(out[1]) == 0 and (kept[1] == -1).all()


def test_evict_lengths_in_place(swa):
    """lens_out may be lens: blocks that start after others have cut a length cut the same tokens."""
    g = _gen(22)
    B, H, D, page, budget, recent = 16, 8, 64, 32, 500, 40
    lens = [0, 1, 499, 500, 501, 900] + [600 + 17 * b for b in range(10)]
    width, room = -(-max(lens) // page), -(-budget // page)
    cache = _cache(swa, g, B * (width + room), H, D, page, spread=6)
    order = _table(g, B, width + room)
    table, dst = order[:, :width].contiguous(), order[:, width:].contiguous()
    pool = ref.pool_of(cache)
    kept, out = ref.evict(pool, table, lens, dst, budget, recent)
    held = _ints(lens)
    gk, go = swa.swa_cache_evict(cache, table, held, dst, budget, recent, lens_out=held)
    swa.swa_check_device()
    assert go is held and torch.equal(held.cpu(), out)
    assert torch.equal(gk.cpu(), kept)
    _same_pool(cache, pool)


# ---- key weights -------------------------------------------------------------------------------

def _ref_lse(q, k, window, causal):
    B, Hq, Lq, D = q.shape
    G, Lk = Hq // k.shape[1], k.shape[2]
    x = q.double().cpu() @ k.double().cpu().repeat_interleave(G, 1).transpose(-1, -2) / math.sqrt(D)
    d = torch.arange(Lq)[:, None] + (Lk - Lq) - torch.arange(Lk)
    see = (d < window) & ((d >= 0) if causal else (d > -window))
    return torch.logsumexp(x.masked_fill(~see, -math.inf), -1).float().cuda()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("B,Hq,H,Lq,Lk,D,window,causal", [
    (1, 1, 1, 1, 1, 64, 1, True),
    (2, 4, 2, 255, 255, 64, 64, True),
    (1, 2, 1, 300, 300, 128, 1, True),
    (1, 2, 2, 512, 512, 128, 512, True),
    (1, 6, 2, 130, 1000, 128, 77, True),
    (1, 4, 1, 700, 700, 256, 200, True),
    (2, 2, 1, 129, 257, 256, 1000, True),
    (1, 4, 2, 333, 400, 64, 50, False),
    (1, 3, 3, 640, 640, 128, 640, False),
    (1, 2, 1, 1, 513, 128, 100, True),
    (1, 2, 1, 1500, 1500, 128, 300, True),
])
def test_key_weights(swa, B, Hq, H, Lq, Lk, D, window, causal, dtype):
    g = _gen(Lq + Lk + D)
    q = torch.randn((B, Hq, Lq, D), generator=g, device="cuda").to(dtype)
    k = torch.randn((B, H, Lk, D), generator=g, device="cuda").to(dtype)
    lse = _ref_lse(q, k, window, causal)
    w, tol = ref.key_weights(q, k, lse, window, causal=causal)
    got = torch.full((B, H, Lk), math.nan, device="cuda")
    swa.swa_attn_key_weights(q, k, lse, window, causal=causal, out=got)
    swa.swa_check_device()
    _near(got, w, tol, "weights")
    # every row gives out one, up to the keys' errors together (lse's rounding is among them)
    total = got.double().cpu().sum(-1)
    assert ((total - (Hq // H) * Lq).abs() <= tol.sum(-1)).all()
    again = swa.swa_attn_key_weights(q, k, lse, window, causal=causal)
    assert torch.equal(again, got)


def test_key_weights_nan_stays_inside_the_window(swa):
    """A NaN query row reaches the keys it sees and no others."""
    g = _gen(31)
    q = torch.randn((1, 2, 400, 128), generator=g, device="cuda").bfloat16()
    k = torch.randn((1, 1, 400, 128), generator=g, device="cuda").bfloat16()
    lse = _ref_lse(q, k, 50, True)
    clean = swa.swa_attn_key_weights(q, k, lse, 50)
    q[0, 1, 200] = math.nan
    lse[0, 0, 300] = math.nan
    got = swa.swa_attn_key_weights(q, k, lse, 50)
    swa.swa_check_device()
    seen = torch.zeros(400, dtype=torch.bool, device="cuda")
    seen[151:201] = True
    seen[251:301] = True
    assert torch.equal(torch.isnan(got[0, 0]), seen)
    assert torch.equal(got[0, 0][~seen], clean[0, 0][~seen])


# ---- a run of them together --------------------------------------------------------------------

def _serve(swa, prompt, steps, budget, window):
    """A prompt through the training forward, its tokens and weights into the cache, tokens one by
    one, an eviction, more tokens: every result against the 64-bit forms on the state the GPU had."""
    g = _gen(41)
    B, Hq, H, D, page = 2, 4, 2, 128, 64
    room = -(-(budget + steps) // page)
    width = -(-(prompt + steps) // page)
    cache = swa.SwaCache.empty(B * (width + room), H, D, page)
    order = _table(g, B, width + room)
    table, spare = order[:, :width].contiguous(), order[:, width:].contiguous()

    def rand(heads, n):
        return torch.randn((B, heads, n, D), generator=g, device="cuda").bfloat16()

    q, k, v = rand(Hq, prompt), rand(H, prompt), rand(H, prompt)
    _, lse = swa.swa_attn_fwd(q, k, v, window)
    w = swa.swa_attn_key_weights(q, k, lse, window)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    swa.swa_cache_append(cache, table, lens, k, v, weight=w)
    want, tol = ref.key_weights(q, k, lse, window)
    stored = torch.stack([torch.stack([
        torch.cat([cache.weight[int(p), h] for p in table[b]])[:prompt] for h in range(H)])
        for b in range(B)])
    _near(stored, want, tol, "prompt weights")
    lens += prompt
    for phase in range(2):
        for _ in range(steps):
            k1, v1, q1 = rand(H, 1), rand(H, 1), rand(Hq, 1)
            pool = ref.pool_of(cache)
            ref.append(pool, table, lens, k1, v1)
            swa.swa_cache_append(cache, table, lens, k1, v1)
            _same_pool(cache, pool)
            o, le, to, tl, tw = ref.attn(pool, table, lens, q1, window, accumulate=True)
            go, gl = swa.swa_cache_attn(q1, cache, table, lens, window, accumulate=True)
            _near(go, o, to, "o")
            _near(gl, le, tl, "lse")
            _near(cache.weight, pool["weight"], tw, "weight")
            lens = lens + 1
        if phase == 0:
            pool = ref.pool_of(cache)
            kept, out = ref.evict(pool, table, lens, spare, budget, 8)
            gk, lens = swa.swa_cache_evict(cache, table, lens, spare, budget, 8)
            assert torch.equal(gk.cpu(), kept) and torch.equal(lens.cpu(), out)
            _same_pool(cache, pool)
            table = spare
    swa.swa_check_device()


def test_serving_full_layer(swa):
    _serve(swa, prompt=300, steps=4, budget=100, window=1 << 20)


def test_serving_sliding_layer(swa):
    _serve(swa, prompt=170, steps=3, budget=150, window=64)


def test_serving_step_in_a_graph(swa):
    """A captured step (append, attention, lengths) replayed equals eager steps bit for bit, while
    other lengths than the captured ones hold, on a stream of its own."""
    g = _gen(51)
    B, Hq, H, D, page, n = 3, 4, 2, 128, 32, 40
    width = 6

    def state():
        gg = _gen(52)
        c = _cache(swa, gg, B * width, H, D, page)
        return c, _table(gg, B, width), _ints([0, 31, 100])

    ks = torch.randn((n, B, H, 1, D), generator=g, device="cuda").bfloat16()
    qs = torch.randn((n, B, Hq, 1, D), generator=g, device="cuda").bfloat16()
    eager = []
    cache, table, lens = state()
    for i in range(n):
        swa.swa_cache_append(cache, table, lens, ks[i], ks[i])
        eager.append(swa.swa_cache_attn(qs[i], cache, table, lens, 64, accumulate=True))
        lens += 1
    weight = cache.weight.clone()
    cache, table, lens = state()
    k, q = ks[0].clone(), qs[0].clone()
    out = torch.empty_like(q)
    lse = torch.empty((B, Hq, 1), device="cuda")
    need = swa.swa_cache_attn_workspace_bytes(B, Hq, H, 1, D, width, page, True)
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        swa.swa_cache_append(cache, table, lens, k, k)
        swa.swa_cache_attn(q, cache, table, lens, 64, accumulate=True, out=out, lse=lse,
                           workspace=ws)
        lens += 1
    for i in range(n):
        k.copy_(ks[i])
        q.copy_(qs[i])
        graph.replay()
        assert torch.equal(out, eager[i][0]) and torch.equal(lse, eager[i][1]), i
    assert torch.equal(weight, cache.weight)
    swa.swa_check_device()


@pytest.mark.parametrize("B,H,page,longest,budget,recent", [
    (1, 2, 64, 70000, 3000, 100),   # a cluster of eight CTAs
    (9, 16, 32, 5000, 700, 0),      # one or two
    (1, 1, 128, 450000, 777, 77),   # slices larger than shared memory holds
])
def test_evict_long(swa, B, H, page, longest, budget, recent):
    """Long sequences against torch's stable sort: the chosen slots, and the weights moved with them."""
    g = _gen(longest)
    D = 64
    width, room = -(-longest // page), -(-budget // page)
    cache = _cache(swa, g, B * (width + room), H, D, page)
    cache.weight.copy_(torch.round(cache.weight * 512) / 512)
    order = _table(g, B, width + room)
    table, dst = order[:, :width].contiguous(), order[:, width:].contiguous()
    lens = [longest - 37 * b for b in range(B)]
    w = cache.weight[table.long()].transpose(1, 2).reshape(B, H, -1).clone()
    kept, out = swa.swa_cache_evict(cache, table, _ints(lens), dst, budget, recent)
    swa.swa_check_device()
    assert out.tolist() == [min(n, budget) for n in lens]
    for b, n in enumerate(lens):
        best = torch.sort(w[b, :, :n - recent], dim=-1, descending=True, stable=True).indices
        want = torch.sort(best[:, :budget - recent], dim=-1).values
        want = torch.cat([want, torch.arange(n - recent, n, device="cuda").expand(H, -1)], 1)
        assert torch.equal(kept[b].long(), want)
        moved = cache.weight[dst[b].long()].transpose(0, 1).reshape(H, -1)[:, :budget]
        assert torch.equal(moved, torch.gather(w[b], 1, want))


# ---- further corners ---------------------------------------------------------------------------

def test_append_fp16_ends(swa):
    """fp16's largest and subnormal numbers, alone and beside older tokens of a far larger scale,
    where the new codes vanish or the old ones do."""
    g = _gen(61)
    D, page = 64, 32
    cache = swa.SwaCache.empty(6, 1, D, page)
    table = _ints([[4, 0, 2, 5, 1, 3]])
    pool = ref.pool_of(cache)

    def put(lens, k, v):
        ref.append(pool, table, lens, k, v)
        swa.swa_cache_append(cache, table, _ints(lens), k, v)
        swa.swa_check_device()
        _same_pool(cache, pool)

    def rand(n, scale, dtype):
        x = torch.randn((1, 1, n, D), generator=g, device="cuda") * scale
        return x.to(dtype)

    put([0], rand(5, 1e4, torch.float16).clamp(-65504, 65504), rand(5, 2.0**-22, torch.float16))
    put([5], rand(5, 2.0**-20, torch.float16), rand(5, 1.0, torch.float16))
    put([10], rand(5, 1e9, torch.bfloat16), rand(5, 1e-12, torch.bfloat16))
    put([15], rand(5, 1.0, torch.float16), rand(5, 6e4, torch.float16).clamp(-65504, 65504))
    put([20], rand(5, 60.0, torch.bfloat16), rand(5, 1e13, torch.bfloat16))
    put([25], rand(60, 2.0**-14, torch.float16), rand(60, 1e-3, torch.float16))
    put([85], rand(20, 1e-20, torch.float32), rand(20, 1e-30, torch.float32))
    edge = torch.tensor([448.0 * 2**-10, 2.0**-24, 3 * 2.0**-24, 2.0**-14, 2.0**-19, 2.0**-20, 0.0, -0.0])
    e = edge.repeat(D // 8).view(1, 1, 1, D).cuda()
    put([105], e.half(), -e.half())


def test_attn_many_sequences(swa):
    """More sequences than one launch takes."""
    g = _gen(62)
    B, width, page, D = 2100, 2, 32, 64
    cache = _cache(swa, g, B * width, 1, D, page)
    table = _table(g, B, width)
    lens = [(7 * i) % 60 for i in range(B)]
    q = torch.randn((B, 2, 1, D), generator=g, device="cuda").bfloat16()
    pool = ref.pool_of(cache)
    o, lse, to, tl, tw = ref.attn(pool, table, lens, q, 40, accumulate=True)
    go, gl = swa.swa_cache_attn(q, cache, table, _ints(lens), 40, accumulate=True)
    swa.swa_check_device()
    _near(go, o, to, "o")
    _near(gl, lse, tl, "lse")
    _near(cache.weight, pool["weight"], tw, "weight")


def test_offsets_past_32_bits(swa):
    """A pool of more than 2^32 bytes: the last pages, through append, attention and eviction."""
    g = _gen(63)
    pages, H, page, D = 34000, 16, 64, 128  # 4.46e9 bytes of keys
    cache = swa.SwaCache.empty(pages, H, D, page)
    last = pages - 8
    table = _ints([[last + 3, last, last + 5], [7, last + 1, 9]])
    dst = _ints([[last + 2, last + 7], [last + 4, 1]])
    T = 150
    k = torch.randn((2, H, T, D), generator=g, device="cuda").bfloat16()
    v = torch.randn((2, H, T, D), generator=g, device="cuda").bfloat16()
    w = torch.rand((2, H, T), generator=g, device="cuda")
    swa.swa_cache_append(cache, table, _ints([0, 0]), k, v, weight=w)
    small = swa.SwaCache.empty(8, H, D, page)
    stable, sdst = _ints([[0, 1, 2], [3, 4, 5]]), _ints([[6, 7], [6, 7]])
    swa.swa_cache_append(small, stable, _ints([0, 0]), k, v, weight=w)
    q = torch.randn((2, 2 * H, 1, D), generator=g, device="cuda").bfloat16()
    lens = _ints([149, 149])
    a = swa.swa_cache_attn(q, cache, table, lens, 1000, accumulate=True)
    b = swa.swa_cache_attn(q, small, stable, lens, 1000, accumulate=True)
    swa.swa_check_device()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    kept, _ = swa.swa_cache_evict(cache, table, _ints([150, 150]), dst, 100, 10)
    skept, _ = swa.swa_cache_evict(small, stable[:1], _ints([150]), sdst[:1], 100, 10)
    swa.swa_check_device()
    assert torch.equal(kept[:1], skept)
    for i in range(2):
        rows = 64 if i == 0 else 36
        for x, y in ((cache.k, small.k), (cache.v, small.v)):
            assert torch.equal(x[int(dst[0, i])].view(torch.uint8)[:, :rows],
                               y[int(sdst[0, i])].view(torch.uint8)[:, :rows])


def test_calls_on_two_streams(swa):
    """Two sequences' steps on two streams at once, each with buffers of its own, equal the same steps
    one after the other."""
    g = _gen(64)
    H, D, page, n = 4, 128, 64, 12

    def state(seed):
        gg = _gen(seed)
        c = _cache(swa, gg, 64, H, D, page)
        return c, _table(gg, 1, 60), _ints([1500 + seed])

    ks = torch.randn((2, n, 1, H, 1, D), generator=g, device="cuda").bfloat16()
    qs = torch.randn((2, n, 1, 3 * H, 1, D), generator=g, device="cuda").half()

    def step(st, i, j):
        c, table, lens = st
        swa.swa_cache_append(c, table, lens, ks[j, i], ks[j, i])
        r = swa.swa_cache_attn(qs[j, i], c, table, lens, 1 << 20, accumulate=True)
        lens += 1
        return r

    want = []
    for j in range(2):
        st = state(j)
        want.append([step(st, i, j) for i in range(n)] + [st[0].weight.clone()])
    states = [state(0), state(1)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    torch.cuda.synchronize()
    for i in range(n):
        for j in range(2):
            with torch.cuda.stream(streams[j]):
                got[j].append(step(states[j], i, j))
    torch.cuda.synchronize()
    swa.swa_check_device()
    for j in range(2):
        for a, b in zip(got[j], want[j]):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        assert torch.equal(states[j][0].weight, want[j][-1])


def test_evict_and_weights_in_a_graph(swa):
    """A captured prompt (forward, key weights, append) and eviction replayed on other inputs."""
    g = _gen(65)
    N, Hq, H, D, page, budget = 500, 4, 2, 64, 32, 100
    cache = swa.SwaCache.empty(40, H, D, page)
    table = torch.arange(16, dtype=torch.int32, device="cuda").view(1, 16)
    dst = torch.arange(20, 24, dtype=torch.int32, device="cuda").view(1, 4)
    zero, full = _ints([0]), _ints([N])

    def draw():
        return [torch.randn((1, h, N, D), generator=g, device="cuda").bfloat16() for h in (Hq, H, H)]

    def run(q, k, v):
        _, lse = swa.swa_attn_fwd(q, k, v, 128)
        w = swa.swa_attn_key_weights(q, k, lse, 128)
        swa.swa_cache_append(cache, table, zero, k, v, weight=w)
        kept, lens = swa.swa_cache_evict(cache, table, full, dst, budget, 16)
        return w, kept, lens

    a, b = draw(), draw()
    want = []
    for x in (a, b):
        r = run(*x)
        want.append([t.clone() for t in r] + [cache.k.view(torch.uint8).clone()])
    held = [t.clone() for t in a]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(*held)
    for x, y in ((a, want[0]), (b, want[1])):
        for h, t in zip(held, x):
            h.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        for p, r in zip(out, y):
            assert torch.equal(p, r)
        assert torch.equal(cache.k.view(torch.uint8), y[-1])
    swa.swa_check_device()


@pytest.mark.parametrize("B,Hq,H,L,D,window", [
    (1, 16, 2, 5000, 128, 700), (1, 8, 8, 3000, 256, 3000), (3, 4, 4, 2049, 64, 100),
    (1, 32, 16, 9000, 128, 1024),
])
def test_key_weights_long(swa, B, Hq, H, L, D, window):
    """Many tasks a pair, full and cut walks, against 64-bit sums on the GPU."""
    g = _gen(L)
    q = torch.randn((B, Hq, L, D), generator=g, device="cuda").bfloat16()
    k = torch.randn((B, H, L, D), generator=g, device="cuda").bfloat16()
    lse = torch.empty((B, Hq, L), device="cuda")
    want = torch.zeros((B, H, L), dtype=torch.float64, device="cuda")
    for b in range(B):
        for h in range(Hq):
            for i in range(0, L, 1024):
                z, lo = min(L, i + 1024), max(0, i - window + 1)
                x = q[b, h, i:z].double() @ k[b, h // (Hq // H), lo:z].double().T / math.sqrt(D)
                d = torch.arange(i, z, device="cuda")[:, None] - torch.arange(lo, z, device="cuda")
                x = x.masked_fill((d < 0) | (d >= window), -math.inf)
                lse[b, h, i:z] = torch.logsumexp(x, -1).float()
                want[b, h // (Hq // H), lo:z] += torch.exp(x - lse[b, h, i:z, None].double()).sum(0)
    got = swa.swa_attn_key_weights(q, k, lse, window)
    swa.swa_check_device()
    # a score is an fp32 sum of D products and a scaling, so off by at most (D + 8) 2^-24 of
    # scale |q| |k| (Cauchy-Schwarz); lse's product with log2(e), the exponential and the sum of the
    # weights (compensated) add a few 2^-21
    es = (D + 8) * 2.0**-24 / math.sqrt(D) * float(q.float().norm(dim=-1).max() *
                                                   k.float().norm(dim=-1).max())
    assert ((got.double() - want).abs() <= (2 * es + 2.0**-18) * want + 1e-30).all()


# ---- arguments ---------------------------------------------------------------------------------

@pytest.mark.parametrize("H_q,H,D,T,lens,dtype", [
    (4, 2, 64, 3, [90, 700], torch.float16),
    (8, 2, 128, 1, [2000, 31], torch.bfloat16),
    (6, 1, 256, 9, [400, 0], torch.bfloat16),
])
@pytest.mark.parametrize("scale", [0.5, 1e-3])
def test_attn_scale_and_output_over_q(swa, H_q, H, D, T, lens, dtype, scale):
    """A scale of the caller's, buffers of the caller's, and o written over q."""
    g = _gen(D + T)
    page, B, window = 32, len(lens), 300
    width = -(-(max(lens) + T) // page)
    cache = _cache(swa, g, B * width, H, D, page, spread=3)
    table = _table(g, B, width)
    q = torch.randn((B, H_q, T, D), generator=g, device="cuda").to(dtype)
    o, lse, to, tl, _ = ref.attn(ref.pool_of(cache), table, lens, q, window, scale=scale)
    lse_out = torch.full((B, H_q, T), math.nan, device="cuda")
    need = swa.swa_cache_attn_workspace_bytes(B, H_q, H, T, D, width, page)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    go, gl = swa.swa_cache_attn(q, cache, table, _ints(lens), window, scale=scale, out=q,
                                lse=lse_out, workspace=ws)
    swa.swa_check_device()
    assert go is q and gl is lse_out
    _near(go, o, to, "o")
    _near(gl, lse, tl, "lse")


@pytest.mark.parametrize("scale", [0.5, 1e-3])
def test_key_weights_scale(swa, scale):
    g = _gen(71)
    q = torch.randn((1, 4, 200, 64), generator=g, device="cuda").to(torch.bfloat16)
    k = torch.randn((1, 2, 333, 64), generator=g, device="cuda").to(torch.bfloat16)
    x = q.double().cpu() @ k.double().cpu().repeat_interleave(2, 1).transpose(-1, -2) * scale
    d = torch.arange(200)[:, None] + 133 - torch.arange(333)
    lse = torch.logsumexp(x.masked_fill((d < 0) | (d >= 90), -math.inf), -1).float().cuda()
    w, tol = ref.key_weights(q, k, lse, 90, scale=scale)
    need = swa.swa_attn_key_weights_workspace_bytes(1, 4, 2, 200, 333, 64, 90)
    ws = torch.full((max(need, 16),), 255, dtype=torch.uint8, device="cuda")
    got = swa.swa_attn_key_weights(q, k, lse, 90, scale=scale, workspace=ws)
    swa.swa_check_device()
    _near(got, w, tol, "weights")


def test_binding_refusals(swa):
    """Tensors of a wrong kind, shape, type or layout raise before anything is launched."""
    cache = swa.SwaCache.empty(8, 2, 64, page=32)
    k = torch.zeros((2, 2, 4, 64), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((2, 4, 1, 64), dtype=torch.bfloat16, device="cuda")
    table, lens = _ints([[0, 1], [2, 3]]), _ints([5, 6])
    dst = _ints([[4], [5]])
    append, attn, evict = swa.swa_cache_append, swa.swa_cache_attn, swa.swa_cache_evict
    weights = swa.swa_attn_key_weights
    wrong = (TypeError, ValueError)
    with pytest.raises(wrong):
        swa.SwaCache(cache.k, cache.v, cache.k_scale.double(), cache.v_scale)
    with pytest.raises(wrong):
        swa.SwaCache(cache.k, cache.v[:7], cache.k_scale, cache.v_scale)
    with pytest.raises(wrong):
        swa.SwaCache(cache.k, cache.v, cache.k_scale, cache.v_scale, cache.weight[..., ::2])
    with pytest.raises(AttributeError):
        cache.k = cache.v
    for t, n in ((table.long(), lens), (table, lens.long()), (table[0], lens), (table, lens[:1]),
                 (table.cpu(), lens), (table.t(), lens)):
        for call in (lambda: append(cache, t, n, k, k), lambda: attn(q, cache, t, n, 9),
                     lambda: evict(cache, t, n, dst, 20, 2)):
            with pytest.raises(wrong):
                call()
    for bad in (k.double(), k[:1], k[:, :1], k[..., :32], k.transpose(1, 2), k.cpu()):
        with pytest.raises(wrong):
            append(cache, table, lens, bad, k)
        with pytest.raises(wrong):
            append(cache, table, lens, k, bad)
    with pytest.raises(wrong):
        append(cache, table, lens, k, k.half())
    with pytest.raises(wrong):
        append(cache, table, lens, k, k, weight=torch.zeros((2, 2, 3), device="cuda"))
    with pytest.raises(wrong):
        append(cache, table, lens, k, k, new=_ints([1]))
    for bad in (q.float(), q[:1], q[..., :32], q.cpu(), q.expand(2, 4, 3, 64)):
        with pytest.raises(wrong):
            attn(bad, cache, table, lens, 9)
    for kw in (dict(out=q.half()), dict(out=q[:, :2]), dict(lse=torch.zeros((2, 4), device="cuda")),
               dict(new=lens.float())):
        with pytest.raises(wrong):
            attn(q, cache, table, lens, 9, **kw)
    for kw in (dict(window=0), dict(window=9, scale=-1.0),
               dict(window=9, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(swa.SwaError):
            attn(q, cache, table, lens, **kw)
    with pytest.raises(wrong):
        evict(cache, table, lens, dst[0], 20, 2)
    with pytest.raises(wrong):
        evict(cache, table, lens, dst, 20, 2, kept=torch.zeros((2, 2, 19), dtype=torch.int32, device="cuda"))
    with pytest.raises(wrong):
        evict(cache, table, lens, dst, 0, 0)
    for budget, recent in ((20, 21), (33, 2)):
        with pytest.raises(swa.SwaError):
            evict(cache, table, lens, dst, budget, recent)
    with pytest.raises(swa.SwaError):
        evict(cache, table, lens, table, 20, 2)
    lse = torch.zeros((2, 4, 1), device="cuda")
    for args in ((q, k[:1], lse), (q, k, lse[..., 0]), (q, k.half(), lse), (q, k, lse.double()),
                 (q, k.cpu(), lse)):
        with pytest.raises(wrong):
            weights(*args, 9)
    with pytest.raises(swa.SwaError):
        weights(q, k, lse, 0)
    torch.cuda.synchronize()
    swa.swa_check_device()
    assert (ref.pool_of(cache)["k"] == 0).all()


def test_elements_need_only_their_own_alignment(swa):
    """Scales, lse and weights that begin one element behind a 16-byte boundary give the same bits."""
    g = _gen(81)
    B, H_q, H, D, page, T = 2, 4, 2, 64, 32, 3
    cache = _cache(swa, g, 8, H, D, page, spread=3)
    table, lens = _table(g, B, 4), _ints([70, 33])
    q = torch.randn((B, H_q, T, D), generator=g, device="cuda").to(torch.bfloat16)
    k = torch.randn((B, H, T, D), generator=g, device="cuda").to(torch.bfloat16)

    def off(x):
        y = torch.zeros(x.numel() + 1, dtype=x.dtype, device="cuda")[1:].view(x.shape)
        return y.copy_(x)

    odd = swa.SwaCache(cache.k.view(torch.uint8).clone().view(torch.float8_e4m3fn),
                       cache.v.view(torch.uint8).clone().view(torch.float8_e4m3fn),
                       off(cache.k_scale), off(cache.v_scale), cache.weight.clone())
    given = torch.rand((B, H, T), generator=g, device="cuda")
    out = []
    for c, move in ((cache, lambda x: x), (odd, off)):
        swa.swa_cache_append(c, move(table), move(lens), k, k, weight=move(given))
        lse = move(torch.zeros((B, H_q, T), device="cuda"))
        o, _ = swa.swa_cache_attn(q, c, move(table), move(lens), 50, accumulate=True, lse=lse)
        w = swa.swa_attn_key_weights(q, k, move(lse), 2, out=move(torch.zeros((B, H, T), device="cuda")))
        spare = [p for p in range(8) if p not in table[:, :3].flatten().tolist()]
        dst = _ints([[spare[0]], [spare[1]]])
        kept, m = swa.swa_cache_evict(c, move(table[:, :3].contiguous()), move(lens), move(dst), 30, 4)
        swa.swa_check_device()
        out.append((o, lse, w, kept, m, *ref.pool_of(c).values()))
    for x, y in zip(*out):
        assert torch.equal(torch.nan_to_num(x, nan=1e9), torch.nan_to_num(y, nan=1e9))
