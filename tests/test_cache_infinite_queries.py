"""A query with an infinite element has infinite or NaN scores, and exp(x - lse) of those is NaN: so are
its answer, its log-sum-exp and the weights that it adds, whatever the scores' signs.  Other rows are
untouched."""
import math

import pytest
import torch

from test_cache import _cache, _gen, _ints, _table

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("D,G,T,lens,window,wide", [
    (64, 2, 1, [0], 5, 0),          # one key: half of the queries below have the score -inf alone
    (128, 4, 1, [0, 1], 1, 0),
    (128, 5, 4, [0, 40], 3, 0),
    (256, 8, 3, [9, 700], 1000, 0),
    (64, 16, 5, [33, 2], 2, 0),
    (128, 8, 5, [1500, 0], 1 << 20, 700000),  # two tiles of rows a warp
])
def test_infinite_queries(swa, dtype, D, G, T, lens, window, wide):
    g = _gen(D + G + T)
    B, page = len(lens), 32
    width = -(-(max(lens) + T) // page)
    cache = _cache(swa, g, B * width, 1, D, page)
    held = _table(g, B, width)
    table = torch.full((B, max(width, wide // page)), -1, dtype=torch.int32, device="cuda")
    table[:, :width] = held
    # no code is zero, so no product is NaN and every score of an infinite query is an infinity
    codes = cache.k.view(torch.uint8)
    codes[(codes & 0x7F) == 0] = 0x38
    q = torch.randn((B, G, T, D), generator=g, device="cuda").to(dtype)
    before = cache.weight.clone()
    o, lse = swa.swa_cache_attn(q, cache, table, _ints(lens), window, accumulate=True)
    plain = cache.weight.clone()
    for sign in (math.inf, -math.inf):
        for b in range(B):
            h, t = (3 * b + 1) % G, T - 1
            bad = q.clone()
            bad[b, h, t, 5] = sign
            cache.weight.copy_(before)
            go, gl = swa.swa_cache_attn(bad, cache, table, _ints(lens), window, accumulate=True)
            swa.swa_check_device()
            hit = torch.zeros((B, G, T), dtype=torch.bool, device="cuda")
            hit[b, h, t] = True
            assert torch.isnan(go[hit].float()).all() and torch.isnan(gl[hit]).all()
            assert torch.equal(go[~hit], o[~hit]) and torch.equal(gl[~hit], lse[~hit])
            at = lens[b] + t
            seen = torch.zeros_like(before, dtype=torch.bool)
            for s in range(max(0, at - window + 1), at + 1):
                seen[int(table[b, s // page]), 0, s % page] = True
            assert torch.isnan(cache.weight[seen]).all()
            assert torch.equal(cache.weight[~seen], plain[~seen])
