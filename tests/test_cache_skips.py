"""What eviction does with sequences and pages that it skips: nothing of theirs is kept or written."""
import pytest
import torch

from test_cache import _cache, _gen, _ints, _table

pytestmark = pytest.mark.gpu


def _bytes(cache):
    return [t.view(torch.uint8).clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale,
                                                  cache.weight)]


@pytest.mark.parametrize("D,page", [(64, 32), (256, 64)])
@pytest.mark.parametrize("bad", [-1, 2**31 - 1, -2**31, "longer"])
@pytest.mark.parametrize("in_place", [False, True])
def test_a_skipped_sequence_keeps_nothing(swa, D, page, bad, in_place):
    g = _gen(D)
    budget = page + 1
    cache = _cache(swa, g, 15, 2, D, page)
    order = _table(g, 3, 5)
    table, dst = order[:, :3].contiguous(), order[:, 3:].contiguous()
    lens = _ints([3 * page, 3 * page + 1 if bad == "longer" else bad, 5])
    before = _bytes(cache)
    kept, out = swa.swa_cache_evict(cache, table, lens, dst, budget, 7, lens_out=lens if in_place else None)
    with pytest.raises(swa.SwaError, match="INDEX"):
        swa.swa_check_device()
    assert out.tolist() == [budget, 0, 5]
    assert (kept[1] == -1).all() and (kept[0] >= 0).all() and (kept[2, :, 5:] == -1).all()
    for was, now in zip(before, _bytes(cache)):
        for p in (*table.flatten().tolist(), *dst[1].tolist()):
            assert torch.equal(was[p], now[p])


def test_skipped_pages(swa):
    """Tokens on a page that is none are the lightest; a place that one of them gets stays as it was."""
    g = _gen(5)
    H, D, page, budget, recent = 2, 128, 32, 40, 8
    cache = _cache(swa, g, 8, H, D, page)
    cache.weight.neg_()  # every real token is below zero
    table, dst = _ints([[3, 8, 1]]), _ints([[0, 6]])
    before = _bytes(cache)
    kept, out = swa.swa_cache_evict(cache, table, _ints([96]), dst, budget, recent)
    with pytest.raises(swa.SwaError, match="INDEX"):
        swa.swa_check_device()
    # 56 of the 88 tokens that compete are real, and 32 of those stay
    assert out.tolist() == [budget] and not ((kept >= 32) & (kept < 64)).any()
    # with more room all real ones stay, and the earliest of the others
    dst3 = _ints([[0, 6, 5]])
    kept, _ = swa.swa_cache_evict(cache, table, _ints([96]), dst3, 70, recent)
    with pytest.raises(swa.SwaError, match="INDEX"):
        swa.swa_check_device()
    assert kept[0, 0].tolist() == list(range(38)) + list(range(64, 96))
    w, k = before[4].view(torch.float32), before[0]
    # slots 32..37 of the destination belong to them: the rows 0..5 of its second page
    f8, f32 = torch.float8_e4m3fn, torch.float32
    cache2 = swa.SwaCache(before[0].clone().view(f8), before[1].clone().view(f8),
                          before[2].clone().view(f32), before[3].clone().view(f32), w.clone())
    swa.swa_cache_evict(cache2, table, _ints([96]), dst3, 70, recent)
    with pytest.raises(swa.SwaError, match="INDEX"):
        swa.swa_check_device()
    assert torch.equal(cache2.weight[6, :, :6], w[6, :, :6])
    assert torch.equal(cache2.k.view(torch.uint8)[6, :, :6], k[6, :, :6])
    assert torch.equal(cache2.weight[6, :, 6:], w[1, :, :26])
    # a destination page that is none: its tokens go nowhere, the others move
    before = _bytes(cache2)
    kept, _ = swa.swa_cache_evict(cache2, _ints([[3, 2, 1]]), _ints([90]), _ints([[0, -1]]), 40, 8)
    with pytest.raises(swa.SwaError, match="INDEX"):
        swa.swa_check_device()
    now = _bytes(cache2)
    for was, is_ in zip(before, now):
        for p in (1, 2, 3, 4, 5, 6, 7):
            assert torch.equal(was[p], is_[p])
    assert not torch.equal(before[4][0], now[4][0])
