"""Sinks through an eviction: with their weights set to infinity they stay, first in every head, and sinks=
means the same tokens before and after."""
import math

import pytest
import torch

from test_cache_sinks import attn_ref, ints, make, near

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,page,sinks,recent", [(64, 32, 4, 20), (128, 64, 33, 1), (256, 32, 60, 40)])
def test_sinks_stay(swa, D, page, sinks, recent):
    B, Hq, H, budget, window = 3, 4, 2, 100, 30
    lens = [400, 100, 163]
    cache, g = make(swa, D, 2 * B * 13, H, D, page)
    order = torch.randperm(2 * B * 13, generator=g, device="cuda").to(torch.int32).view(2, B, 13)
    table, spare = order[0].contiguous(), order[1].contiguous()
    first = torch.arange(sinks, device="cuda")
    for b in range(B):
        cache.weight[table[b].long()[first // page], :, first % page] = 1e-9  # lighter than any other
    kept, _ = swa.swa_cache_evict(cache, table, ints(lens), spare, budget, recent)
    lost = [b for b in range(B) if lens[b] > budget]
    assert all(kept[b, h, 0] >= sinks for b in lost for h in range(H))
    for b in range(B):
        cache.weight[table[b].long()[first // page], :, first % page] = math.inf
    kept, left = swa.swa_cache_evict(cache, table, ints(lens), spare, budget, recent)
    swa.swa_check_device()
    assert (kept[:, :, :sinks] == first.int()).all()
    for b in range(B):
        page_of = spare[b].long()[first // page]
        assert torch.isinf(cache.weight[page_of, :, first % page]).all()
    # the last survivor asks over what is left; then its weight is added, and the sinks' stays
    q = torch.randn((B, Hq, 1, D), generator=g, device="cuda").bfloat16()
    at = [min(n, budget) - 1 for n in lens]
    o, lse, _, to, tl, _ = attn_ref(cache, spare, at, q, window, sinks)
    got = swa.swa_cache_attn(q, cache, spare, left - 1, window, sinks=sinks, accumulate=True)
    swa.swa_check_device()
    near(got[0], o, to, "o")
    near(got[1], lse, tl, "lse")
    for b in range(B):
        assert torch.isinf(cache.weight[spare[b].long()[first // page], :, first % page]).all()
