"""Cache attention over a shared prefix reads only what some sequence sees: table entries of pages that none
sees may be -1 or name pages that hold something else by now, and slots that none sees may hold anything.
Against the definition in 64 bits (test_cache_sinks.attn_ref), which looks up visible slots alone."""
import math

import pytest
import torch

from test_cache_shared import setup
from test_cache_sinks import attn_ref, ints, near

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16

CASES = [
    # D, page, T, shared, lens, window, sinks, dtype
    (64, 32, 1, 40, [1290, 1300, 1281], 100, 4, BF16),     # between the sinks and the windows
    (128, 32, 2, 40, [1290, 1300, 1281], 100, 4, BF16),
    (256, 32, 1, 40, [1290, 1300, 1281], 100, 4, FP16),
    (128, 64, 1, 20, [1290, 1300, 1281], 150, 65, BF16),
    (64, 32, 2, 24, [770, 800], 65, 0, BF16),              # before every window, in its first chunk
    (128, 32, 1, 24, [770, 800], 90, 0, FP16),
    (256, 64, 1, 12, [770, 800], 90, 0, BF16),
    (64, 32, 1, 30, [40, 33, 70], 4000, 0, BF16),          # behind the last token of all
    (128, 32, 2, 30, [40, 33, 190], 4000, 0, BF16),
    (256, 32, 1, 30, [40, 33, 90], 4000, 0, FP16),
    (128, 64, 1, 30, [40, 10, 20], 30, 3, BF16),
    (64, 32, 1, 60, [100, 1950, 1930], 80, 0, BF16),       # between one's last token and the others' windows
    (128, 32, 2, 60, [100, 1950, 1930], 80, 33, BF16),
    (256, 32, 1, 60, [100, 900, 1930], 80, 5, FP16),
    (128, 64, 3, 30, [70, 900, 1930], 80, 0, BF16),
    (128, 32, 1, 60, [0, 1950, 500], 1, 0, BF16),          # each itself alone
]


def seen_slots(lens, T, window, sinks, slots):
    seen = torch.zeros(slots, dtype=torch.bool)
    for n in lens:
        for t in range(T):
            p = torch.arange(min(n + t + 1, slots))
            seen[p[(n + t - p < window) | (p < sinks)]] = True
    return seen


def problem(swa, D, page, T, shared, lens, window, sinks, dtype):
    B, Hq, H = len(lens), 4, 2
    width = max(shared + 1, -(-(max(lens) + T) // page))
    cache, table, g = setup(swa, D + page + T, B, H, D, page, shared, width)
    q = torch.randn((B, Hq, T, D), generator=g, device="cuda").to(dtype)
    seen = seen_slots(lens, T, window, sinks, shared * page).view(shared, page)
    return cache, table, q, seen, attn_ref(cache, table, lens, q, window, sinks)


def check(swa, cache, table, lens, q, window, sinks, shared, want):
    o, lse, _, to, tl, _ = want
    got = swa.swa_cache_attn(q, cache, table, ints(lens), window, sinks=sinks, shared=shared)
    swa.swa_check_device()
    near(got[0], o, to, "o")
    near(got[1], lse, tl, "lse")
    return got


@pytest.mark.parametrize("D,page,T,shared,lens,window,sinks,dtype", CASES)
def test_entries_that_nobody_sees(swa, D, page, T, shared, lens, window, sinks, dtype):
    cache, table, q, seen, want = problem(swa, D, page, T, shared, lens, window, sinks, dtype)
    whole = check(swa, cache, table, lens, q, window, sinks, shared, want)
    unseen = ~seen.any(1)
    assert unseen.any()
    table[:, :shared][:, unseen.cuda()] = -1
    got = check(swa, cache, table, lens, q, window, sinks, shared, want)
    assert all(torch.equal(a, b) for a, b in zip(got, whole))


@pytest.mark.parametrize("junk", ["large", "nan"])
@pytest.mark.parametrize("D,page,T,shared,lens,window,sinks,dtype", CASES)
def test_pages_and_slots_that_nobody_sees(swa, D, page, T, shared, lens, window, sinks, dtype, junk):
    cache, table, q, seen, want = problem(swa, D, page, T, shared, lens, window, sinks, dtype)
    pages = table[0, :shared].long()
    for codes in (cache.k, cache.v):  # slots: a NaN each
        x = codes.view(torch.uint8)
        x[pages] = torch.where(seen.cuda()[:, None, :, None], x[pages], 0x7F)
    unseen = pages[~seen.any(1).cuda()]
    for scale in (cache.k_scale, cache.v_scale):  # pages of another use: scales too
        scale[unseen] = 2.0**40 if junk == "large" else math.nan
    check(swa, cache, table, lens, q, window, sinks, shared, want)


def test_a_part_that_begins_where_nobody_sees(swa):
    """Parts of some four hundred chunks, which begin between a short sequence's end and the others' windows:
    the values behind keep their bits, however small their scale."""
    B, H, G, D, page, shared, window = 1024, 1, 16, 64, 128, 512, 1000
    cache, table, g = setup(swa, 3, B, H, D, page, shared, shared + 1)
    cache.v_scale[:] = 2.0**-30
    lens = [100 if b % 8 == 0 else shared * page + b % 90 for b in range(B)]
    q = torch.randn((B, G, 1, D), generator=g, device="cuda").bfloat16()
    table[:, 1:shared - 9] = -1
    got = swa.swa_cache_attn(q, cache, table, ints(lens), window, shared=shared)
    swa.swa_check_device()
    pick = [0, 1, 7, 8, 500, 511, 512, 1016, 1023]
    o, lse, _, to, tl, _ = attn_ref(cache, table[pick], [lens[b] for b in pick], q[pick], window, 0)
    # (the tolerance's 2^-25 of a value counts values of this scale)
    near(got[0][pick], o, to, "o")
    near(got[1][pick], lse, tl, "lse")
