"""Cache attention of a batch whose tables begin with the same pages, on the GPU, against the definition in
64 bits (test_cache_sinks.attn_ref), which knows nothing of sharing: the result is the same."""
import math

import pytest
import torch

from test_cache_sinks import attn_ref, ints, make, near

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16


def setup(swa, seed, B, H, D, page, shared, width, spread=3):
    cache, g = make(swa, seed, shared + B * (width - shared) + 1, H, D, page, spread, weight=False)
    order = torch.randperm(cache.k.shape[0] - 1, generator=g, device="cuda").to(torch.int32)
    table = torch.cat([order[:shared].expand(B, shared), order[shared:].view(B, width - shared)], 1)
    return cache, table.contiguous(), g


CASES = [
    # B, Hq, H, D, page, T, shared, lens behind the prefix (negative: inside it), window, sinks, new, dtype
    (2, 1, 1, 64, 32, 1, 1, [0, 3], 0, 0, None, BF16),
    (2, 2, 2, 128, 64, 1, 2, [0, 100], 0, 0, None, BF16),
    (3, 4, 2, 128, 64, 1, 5, [1, 63, 64], 0, 0, None, FP16),
    (4, 8, 2, 128, 32, 3, 9, [0, 31, 200, 7], 0, 0, [3, 0, 2, 1], BF16),
    (40, 8, 2, 128, 64, 2, 7, list(range(0, 200, 5)), 0, 0, None, BF16),      # tiles cut sequences
    (33, 7, 1, 64, 128, 1, 3, list(range(33)), 0, 0, None, BF16),
    (5, 3, 1, 256, 32, 5, 11, [0, 1, 90, 33, 64], 0, 0, [5, 1, 2, 3, 4], FP16),
    (30, 16, 1, 256, 128, 1, 4, list(range(0, 300, 10)), 0, 0, None, BF16),
    (3, 2, 1, 128, 64, 1, 6, [-384, -200, -1], 0, 0, None, BF16),             # shorter than the prefix
    (4, 4, 2, 64, 64, 2, 6, [-300, 50, -2, 400], 0, 0, [2, 2, 1, 0], BF16),
    (4, 4, 1, 128, 64, 1, 8, [0, 100, 200, 400], 300, 0, None, BF16),         # a window into the prefix
    (4, 4, 1, 128, 64, 2, 8, [100, 200, 300, 500], 90, 0, None, BF16),        # and past all of it
    (4, 4, 1, 128, 64, 2, 8, [100, 200, 300, 500], 90, 70, None, FP16),       # with sinks
    (3, 2, 2, 256, 32, 1, 10, [50, -100, 300], 120, 33, None, BF16),
    (3, 2, 1, 64, 32, 1, 2, [200, 400, 30], 50, 130, None, BF16),             # sinks past the prefix
    (70, 4, 1, 128, 32, 2, 20, [13 * i % 300 for i in range(70)], 500, 4, None, BF16),
    (2, 2, 1, 128, 64, 1, 4, [0, 0], 1, 0, None, BF16),                       # itself alone
    (2, 4, 1, 128, 64, 64, 5, [0, -100], 0, 0, [64, 33], FP16),               # many rows each
]


@pytest.mark.parametrize("B,Hq,H,D,page,T,shared,behind,window,sinks,new,dtype", CASES)
def test_attn(swa, B, Hq, H, D, page, T, shared, behind, window, sinks, new, dtype):
    lens = [shared * page + n for n in behind]
    width = max(shared + 1, -(-(max(lens) + T) // page))
    cache, table, g = setup(swa, B * 100 + T, B, H, D, page, shared, width)
    q = torch.randn((B, Hq, T, D), generator=g, device="cuda").to(dtype)
    W = window or width * page
    o, lse, _, to, tl, _ = attn_ref(cache, table, lens, q, W, sinks, new)
    kw = dict(new=ints(new), sinks=sinks, shared=shared)
    got = swa.swa_cache_attn(q, cache, table, ints(lens), W, **kw)
    swa.swa_check_device()
    near(got[0], o, to, "o")
    near(got[1], lse, tl, "lse")
    again = swa.swa_cache_attn(q, cache, table, ints(lens), W, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_long_prefix(swa):
    """A part of the list spans items, and every part many chunks; scores that rise along the prefix move the
    maximum."""
    B, Hq, H, D, page, shared = 6, 8, 2, 128, 64, 300
    cache, table, g = setup(swa, 5, B, H, D, page, shared, shared + 2)
    lens = [shared * page + 7 * b for b in range(B)]
    rise = torch.linspace(-6, 2, shared, device="cuda").round()
    cache.k_scale[table[0, :shared].long()] = torch.exp2(rise - 6)[:, None].expand(-1, H)
    q = torch.randn((B, Hq, 1, D), generator=g, device="cuda").bfloat16()
    W = (shared + 2) * page
    o, lse, _, to, tl, _ = attn_ref(cache, table, lens, q, W, 0)
    got = swa.swa_cache_attn(q, cache, table, ints(lens), W, shared=shared)
    swa.swa_check_device()
    near(got[0], o, to, "o")
    near(got[1], lse, tl, "lse")


@pytest.mark.parametrize("D,page", [(128, 32), (64, 128), (256, 64)])
def test_value_scales_far_apart(swa, D, page):
    """The documented error: 2^-25 of the largest scale among the shared slots, beside the usual one."""
    B, shared = 3, 8 * 128 // page
    cache, table, g = setup(swa, 6, B, 1, D, page, shared, shared + 1)
    e = torch.randint(-30, 20, (cache.k.shape[0], 1), generator=g, device="cuda").float()
    cache.v_scale[:] = torch.exp2(e)
    lens = [shared * page + b for b in range(B)]
    q = torch.randn((B, 2, 1, D), generator=g, device="cuda").bfloat16()
    W = (shared + 1) * page
    o, lse, _, to, tl, _ = attn_ref(cache, table, lens, q, W, 0)
    got = swa.swa_cache_attn(q, cache, table, ints(lens), W, shared=shared)
    swa.swa_check_device()
    top = cache.v_scale[table[0, :shared].long()].max().item()
    near(got[0], o, to + 2.0**-25 * top, "o")
    near(got[1], lse, tl, "lse")


def test_extreme_queries_and_tokens(swa):
    """Queries of all magnitudes; one with an infinity answers NaN, beside others that do not notice; a token
    whose key is NaN reaches every query that sees it, and none under a window that does not."""
    B, H, D, page, shared = 4, 1, 128, 64, 4
    cache, table, g = setup(swa, 7, B, H, D, page, shared, shared + 1)
    lens = [shared * page + 3 * b for b in range(B)]
    q = torch.randn((B, 2, 1, D), generator=g, device="cuda")
    q[0, 0] *= 2.0**-90
    q[1] = 0.0
    q = q.bfloat16()
    W = (shared + 1) * page
    o, lse, _, to, tl, _ = attn_ref(cache, table, lens, q, W, 0)
    bad = q.clone()
    bad[2, 1, 0, 5] = math.inf
    bad[2, 0, 0, 9] = math.nan
    for qq in (q, bad):
        got = swa.swa_cache_attn(qq, cache, table, ints(lens), W, shared=shared)
        swa.swa_check_device()
        rows = [0, 1, 3] if qq is bad else [0, 1, 2, 3]
        near(got[0][rows], o[rows], to[rows], "o")
        near(got[1][rows], lse[rows], tl[rows], "lse")
        if qq is bad:
            assert torch.isnan(got[0][2]).all() and torch.isnan(got[1][2]).all()
    clean = swa.swa_cache_attn(q, cache, table, ints(lens), 100, shared=shared)
    page0 = int(table[0, 0])
    cache.k.view(torch.uint8)[page0, 0, 20] = 0x7F
    cache.v.view(torch.uint8)[page0, 0, 20] = 0
    got = swa.swa_cache_attn(q, cache, table, ints(lens), W, shared=shared)
    assert torch.isnan(got[0]).all() and torch.isnan(got[1]).all()
    cache.v.view(torch.uint8)[page0, 0, 20] = 0x7F
    got = swa.swa_cache_attn(q, cache, table, ints(lens), 100, shared=shared)
    swa.swa_check_device()
    assert all(torch.equal(a, b) for a, b in zip(got, clean))


def test_only_the_first_table_names_the_prefix_and_one_sequence_shares_nothing(swa):
    B, H, D, page, shared = 3, 2, 64, 32, 6
    cache, table, g = setup(swa, 8, B, H, D, page, shared, shared + 2)
    lens = ints([shared * page + 5 * b for b in range(B)])
    q = torch.randn((B, 4, 1, D), generator=g, device="cuda").bfloat16()
    want = swa.swa_cache_attn(q, cache, table, lens, 256, shared=shared)
    other = table.clone()
    other[1:, :shared] = -1
    got = swa.swa_cache_attn(q, cache, other, lens, 256, shared=shared)
    swa.swa_check_device()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    one = swa.swa_cache_attn(q[1:2].contiguous(), cache, table[1:2].contiguous(), lens[1:2], 256,
                             shared=shared)
    plain = swa.swa_cache_attn(q[1:2].contiguous(), cache, table[1:2].contiguous(), lens[1:2], 256)
    assert all(torch.equal(a, b) for a, b in zip(one, plain))


def test_bad_pages_and_lengths_are_skipped_and_reported(swa):
    B, H, D, page, shared = 4, 1, 128, 32, 9
    cache, table, g = setup(swa, 9, B, H, D, page, shared, shared + 1)
    lens = [shared * page + b for b in range(B)]
    q = torch.randn((B, 2, 1, D), generator=g, device="cuda").bfloat16()
    W = (shared + 1) * page
    holed = table.clone()
    holed[0, 3] = cache.k.shape[0]
    got = swa.swa_cache_attn(q, cache, holed, ints(lens), W, shared=shared)
    with pytest.raises(swa.SwaError, match="INDEX"):
        swa.swa_check_device()
    # the same without that page's tokens: its keys as far away as a masked one
    ref = attn_ref(cache, table, lens, q, W, 0)
    k, v = cache.k.float(), cache.v.float()
    keep = [s for s in range(W) if s // page != 3]
    for b in range(B):
        s = torch.tensor([i for i in keep if i <= lens[b]], device="cuda")
        p = table[b].long()[s // page]
        kk = (k[p, 0, s % page] * cache.k_scale[p, 0, None]).double()
        vv = (v[p, 0, s % page] * cache.v_scale[p, 0, None]).double()
        x = q[b, :, 0].double() @ kk.T / math.sqrt(D)
        r = torch.softmax(x, -1) @ vv
        assert ((got[0][b, :, 0].double() - r).abs() <= 2 * ref[3][b, :, 0]).all()
        assert (got[1][b, :, 0].double() - torch.logsumexp(x, -1)).abs().max() <= 1e-5
    for bad in (-1, 10 * page + 1):
        off = list(lens)
        off[2] = bad
        got = swa.swa_cache_attn(q, cache, table, ints(off), W, shared=shared)
        with pytest.raises(swa.SwaError, match="INDEX"):
            swa.swa_check_device()
        assert not got[0][2].any() and (got[1][2] == -math.inf).all()
        rows = [0, 1, 3]
        near(got[0][rows], ref[0][rows], ref[3][rows], "o")


def test_more_sequences_than_one_launch(swa):
    B, H, D, page, shared = 2500, 1, 64, 32, 3
    cache, table, g = setup(swa, 10, B, H, D, page, shared, shared + 1)
    lens = [shared * page + b % 31 for b in range(B)]
    q = torch.randn((B, 1, 1, D), generator=g, device="cuda").bfloat16()
    W = (shared + 1) * page
    got = swa.swa_cache_attn(q, cache, table, ints(lens), W, shared=shared)
    want = swa.swa_cache_attn(q, cache, table, ints(lens), W)
    swa.swa_check_device()
    # both round p and o once each: 2^-11 and 2^-9, twice
    assert (got[0].double() - want[0].double()).norm() <= 2.0**-7 * want[0].double().norm()
    assert (got[1] - want[1]).abs().max() <= 1e-5
    pick = [0, 1, 511, 1023, 1024, 2047, 2048, 2499]
    o, lse, _, to, tl, _ = attn_ref(cache, table[pick], [lens[b] for b in pick], q[pick], W, 0)
    near(got[0][pick], o, to, "o")
    near(got[1][pick], lse, tl, "lse")


def test_given_buffers_graphs_and_streams(swa):
    B, Hq, H, D, page, shared, T = 5, 8, 2, 128, 64, 10, 2
    cache, table, g = setup(swa, 11, B, H, D, page, shared, shared + 3)
    q = torch.randn((B, Hq, T, D), generator=g, device="cuda").bfloat16()
    lens, W = ints([shared * page + 9 * b for b in range(B)]), 400
    kw = dict(sinks=3, shared=shared)
    need = swa.swa_cache_attn_workspace_bytes(B, Hq, H, T, D, shared + 3, page, window=W, **kw)
    guard = torch.full((need + 64,), 9, dtype=torch.uint8, device="cuda")
    out = q.clone()
    got = swa.swa_cache_attn(out, cache, table, lens, W, out=out, workspace=guard[:need], **kw)  # over q
    want = swa.swa_cache_attn(q, cache, table, lens, W, **kw)
    swa.swa_check_device()
    assert got[0] is out and all(torch.equal(a, b) for a, b in zip(got, want))
    assert (guard[need:] == 9).all()
    with pytest.raises(swa.SwaError, match="WORKSPACE"):
        swa.swa_cache_attn(q, cache, table, lens, W, workspace=guard[:need - 1], **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = swa.swa_cache_attn(q, cache, table, lens, W, **kw)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(other, want))
    later = lens + 30
    after = swa.swa_cache_attn(q, cache, table, later, W, **kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        played = swa.swa_cache_attn(q, cache, table, lens, W, **kw)
    lens += 30
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    swa.swa_check_device()
    assert all(torch.equal(a, b) for a, b in zip(played, after))
