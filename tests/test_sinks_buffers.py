"""Gradients with sinks that would be written over what other kernels of the call still read are refused."""
import pytest
import torch

import sliding_window_flash_gb300 as swa_pkg

INVALID = 1
B, Hq, Hkv, Lq, Lk, D, W, S = 1, 4, 2, 200, 300, 64, 30, 4
ROWS, KEYS, LSE = B * Hq * Lq * D * 2, B * Hkv * Lk * D * 2, B * Hq * Lq * 4
SIZES = dict(q=ROWS, k=KEYS, v=KEYS, o=ROWS, do=ROWS, lse=LSE, dq=ROWS, dk=KEYS, dv=KEYS)
GRADS = ("dq", "dk", "dv")
# (gradient, what it lies over, bytes behind that one's start)
PAIRS = [(a, b, at) for a in GRADS for b in SIZES if b not in ("o", a)
         for at in (0, SIZES[b] - 16, 16 - SIZES[a])]


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("grad,over,at", PAIRS)
def test_refused(grad, over, at, dtype):
    """Addresses that are never followed: the call is refused before anything is launched."""
    place = {name: (i + 1) << 24 for i, name in enumerate(SIZES)}
    place[grad] = place[over] + at
    rc = swa_pkg.load().swa_attn_bwd_sinks(*place.values(), B, Hq, Hkv, Lq, Lk, D, W, S, 1, 0.125, dtype,
                                           1 << 40, 1 << 30, None)
    assert rc == INVALID


@pytest.mark.gpu
def test_the_binding_refuses_it_and_gradients_may_replace_o(swa):
    g = torch.Generator(device="cuda").manual_seed(1)
    q, do = (torch.randn((B, Hq, Lq, D), generator=g, device="cuda").bfloat16() for _ in range(2))
    k, v = (torch.randn((B, Hkv, Lk, D), generator=g, device="cuda").bfloat16() for _ in range(2))
    o, lse = swa.swa_attn_fwd(q, k, v, W, sinks=S)
    want = swa.swa_attn_bwd(q, k, v, o, do, lse, W, sinks=S)
    for kw in (dict(dq=q), dict(dq=do), dict(dk=k), dict(dv=k), dict(dk=want[1], dv=want[1])):
        with pytest.raises(swa.SwaError, match="INVALID"):
            swa.swa_attn_bwd(q, k, v, o, do, lse, W, sinks=S, **kw)
    got = swa.swa_attn_bwd(q, k, v, o, do, lse, W, sinks=S, dq=o)
    swa.swa_check_device()
    assert got[0] is o and all(torch.equal(a, b) for a, b in zip(got, want))
    # no sinks behind the window: the call without them, over q as ever
    every = swa.swa_attn_bwd(q, k, v, o, do, lse, Lk, sinks=S)
    mine = q.clone()
    over = swa.swa_attn_bwd(mine, k, v, o, do, lse, Lk, sinks=S, dq=mine)
    assert over[0] is mine and all(torch.equal(a, b) for a, b in zip(over, every))
