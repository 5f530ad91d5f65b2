"""GPU forward where single rows' scores rise by much after their first key blocks, so that some rows of a
warp, and not the others, leave the one-pass softmax: against a dense softmax in 64 bits.

Rows of a tile are given a direction u; keys from 256 on lie along u.  A rise of 5 makes a block's sum
128 e^5 > 2^12 while the maximum moves by less than 2^8; one of 20 moves the maximum too.  Bars: |LSE
difference| <= 1e-3, norm-wise relative error of O <= 1e-2, as elsewhere.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rise", [5.0, 20.0])
@pytest.mark.parametrize("D,Hq", [(64, 1), (128, 1), (128, 2), (256, 1), (256, 2)])
@pytest.mark.parametrize("rows", [[300], [301, 309], [256, 383], list(range(272, 280)), list(range(512, 640, 3))],
                         ids=lambda r: f"{r[0]}x{len(r)}")
def test_rows_that_rise_alone(swa, D, Hq, rows, rise):
    N = 700
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn((1, Hq, N, D), generator=g, device="cuda") * 0.5
    k = torch.randn((1, 1, N, D), generator=g, device="cuda") * 0.5
    v = torch.randn((1, 1, N, D), generator=g, device="cuda").bfloat16()
    u = torch.zeros(D, device="cuda")
    u[::2] = 1.0
    q[..., ::2] = 0.0                       # other rows do not see u
    q[:, -1, rows] = u
    k[:, :, 256:, ::2] = 0.0
    k[:, :, 256:] += u * (rise * math.sqrt(D) / (D / 2))
    k[:, :, :256, ::2] = 0.0
    q, k = q.bfloat16(), k.bfloat16()
    o, lse = swa.swa_attn_fwd(q, k, v, N)
    swa.swa_check_device()
    see = torch.ones((N, N), dtype=torch.bool, device="cuda").tril()
    x = torch.where(see, q[0].double() @ k[0, 0].double().T / math.sqrt(D), -math.inf)
    ref = torch.softmax(x, -1) @ v[0, 0].double()
    assert (lse[0].double() - torch.logsumexp(x, -1)).abs().max().item() <= 1e-3
    assert (o[0].double() - ref).norm().item() <= 1e-2 * ref.norm().item()
    part = ref[-1, rows]
    assert (o[0, -1, rows].double() - part).norm().item() <= 1e-2 * part.norm().item()
