"""Weights accumulated beside rows that are NaN: a row that sees a token stored as NaN, or whose query
is NaN, gives NaN to the weight of every token that it sees and nothing to any other."""
import math

import pytest
import torch

import cache_ref as ref
from test_cache import _cache, _gen, _ints, _near, _table

pytestmark = pytest.mark.gpu

CASES = [
    # B, Hq, H, D, page, T, lens, window, new, NaN tokens (sequence, slot), NaN queries (b, head, t), dtype
    (1, 2, 1, 64, 32, 1, [40], 8, None, [(0, 38)], [], torch.bfloat16),
    # the third of four new tokens; the first two rows do not see it
    (1, 4, 2, 128, 64, 4, [70], 20, None, [(0, 72)], [], torch.float16),
    # seen by no row: before the window, in its first chunk
    (1, 2, 2, 256, 32, 2, [90], 10, None, [(0, 80)], [], torch.bfloat16),
    # a NaN query in one head of two, of the second sequence only
    (2, 4, 2, 128, 32, 3, [100, 33], 33, None, [], [(1, 3, 1)], torch.bfloat16),
    # more rows than a warp's tile, than two, than a team's
    (2, 12, 2, 64, 64, 5, [200, 150], 70, [5, 3], [(0, 190)], [(1, 0, 2)], torch.bfloat16),
    (1, 8, 1, 128, 64, 9, [300], 90, None, [(0, 304)], [], torch.float16),
    (1, 24, 2, 64, 32, 8, [260], 1000, None, [(0, 263)], [(0, 5, 0)], torch.bfloat16),
    # many parts an item
    (1, 4, 1, 256, 128, 2, [5000], 4000, None, [(0, 5001)], [], torch.bfloat16),
]


def _check(swa, cache, table, lens, q, window, new, tokens, queries):
    for b, s in tokens:  # as append stores them
        page = cache.page
        cache.k.view(torch.uint8)[int(table[b, s // page]), :, s % page] = ref.E4M3_NAN
        cache.v.view(torch.uint8)[int(table[b, s // page]), :, s % page] = 0
    for b, h, t in queries:
        q[b, h, t, 7] = math.nan
    pool = ref.pool_of(cache)
    o, lse, to, tl, tw = ref.attn(pool, table, lens, q, window, new=new, accumulate=True)
    go, gl = swa.swa_cache_attn(q, cache, table, _ints(lens), window, new=_ints(new), accumulate=True)
    swa.swa_check_device()
    _near(go, o, to, "o")
    _near(gl, lse, tl, "lse")
    _near(cache.weight, pool["weight"], tw, "weight")


@pytest.mark.parametrize("B,H_q,H,D,page,T,lens,window,new,tokens,queries,dtype", CASES)
def test_weights_beside_nan_rows(swa, B, H_q, H, D, page, T, lens, window, new, tokens, queries, dtype):
    g = _gen(sum(lens) + D)
    width = -(-(max(lens) + T) // page) + 1
    cache = _cache(swa, g, B * width, H, D, page, spread=3)
    table = _table(g, B, width)
    q = torch.randn((B, H_q, T, D), generator=g, device="cuda").to(dtype)
    _check(swa, cache, table, lens, q, window, new, tokens, queries)


def test_weights_beside_nan_rows_long_tables(swa):
    """The same where a warp has two tiles of rows (a table for long sequences)."""
    g = _gen(91)
    B, H_q, H, D, page, T, lens = 2, 8, 1, 128, 64, 5, [1500, 65]
    width = -(-(max(lens) + T) // page)
    cache = _cache(swa, g, B * width, H, D, page, spread=3)
    table = torch.full((B, 700000 // page), -1, dtype=torch.int32, device="cuda")
    table[:, :width] = _table(g, B, width)
    q = torch.randn((B, H_q, T, D), generator=g, device="cuda").bfloat16()
    _check(swa, cache, table, lens, q, 1 << 20, None, [(0, 1502)], [(1, 2, 3)])


def test_weights_after_an_appended_nan_token(swa):
    """Through append: the weights of the tokens that nobody with a NaN answer sees keep their bits."""
    g = _gen(92)
    D, page, window = 64, 32, 8
    cache = swa.SwaCache.empty(3, 1, D, page)
    table = _ints([[2, 0, 1]])
    k = torch.randn((1, 1, 41, D), generator=g, device="cuda").bfloat16()
    w = torch.rand((1, 1, 41), generator=g, device="cuda")
    k[0, 0, 38, 5] = math.inf
    swa.swa_cache_append(cache, table, _ints([0]), k, k, weight=w)
    q = torch.randn((1, 2, 1, D), generator=g, device="cuda").bfloat16()
    swa.swa_cache_attn(q, cache, table, _ints([40]), window, accumulate=True)
    swa.swa_check_device()
    now = torch.cat([cache.weight[2, 0], cache.weight[0, 0]])
    assert torch.isnan(now[33:41]).all()
    assert torch.equal(now[:33], w[0, 0, :33])
    assert (now[41:] == 0).all()
