"""GPU parity of training attention with sinks (the first S keys visible to every query behind them)
against a dense masked softmax in 64 bits.

Bars as for the other training paths: norm-wise relative error <= 1e-2 for O, dQ, dK, dV, each also on
the sinks' rows of dK and dV alone, and |LSE difference| <= 1e-3.  Where they come from: P, dS and the
results are rounded to 16 bits (half a step is 2^-8 of a bf16 value), at most three such roundings meet in
one number, and independent ones add up as squares: 2^-8 sqrt(3) = 0.0068.
"""
import dataclasses
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

REL, LSE = 1e-2, 1e-3
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@dataclasses.dataclass(frozen=True)
class Shape:
    B: int
    Hq: int
    Hkv: int
    Lq: int
    Lk: int
    D: int
    W: int
    S: int
    causal: bool = True
    dtype: torch.dtype = BF16

    def name(self):
        return "_".join(f"{k}{str(v).replace('torch.', '')}" for k, v in dataclasses.asdict(self).items())


SHAPES = [
    Shape(1, 1, 1, 1, 2, 64, 1, 1),             # one query: itself and a sink
    Shape(1, 2, 1, 17, 17, 128, 3, 40),         # more sinks than keys
    Shape(2, 4, 2, 300, 300, 64, 64, 4),        # far sinks from the second query tile on
    Shape(1, 3, 1, 700, 700, 128, 130, 1),      # an odd number of query heads: one CTA a tile
    Shape(1, 3, 1, 517, 517, 64, 1, 7),         # itself and the sinks alone
    Shape(2, 4, 2, 255, 1000, 128, 64, 127),    # queries a suffix
    Shape(1, 2, 1, 255, 1000, 128, 64, 128),    # sinks end with a block
    Shape(1, 2, 1, 255, 1000, 64, 64, 129),
    Shape(1, 8, 1, 130, 900, 128, 500, 600),    # sinks reach into the window
    Shape(1, 4, 2, 900, 900, 128, 100, 300),    # several blocks of sinks, some of them whole
    Shape(1, 2, 1, 1, 1300, 128, 5, 140),       # one query, a long way from its sinks
    Shape(1, 2, 2, 640, 640, 64, 64, 30, causal=False),
    Shape(1, 4, 2, 300, 777, 128, 33, 130, causal=False),
    Shape(1, 4, 2, 700, 700, 128, 130, 5, dtype=FP16),
    Shape(1, 1, 1, 300, 500, 64, 40, 3, dtype=FP16),
    Shape(1, 2, 1, 700, 700, 256, 130, 5),      # D = 256 on pairs
    Shape(1, 3, 1, 300, 900, 256, 64, 129, dtype=FP16),
    Shape(1, 1, 1, 515, 515, 256, 1, 300),
    Shape(2, 2, 1, 400, 400, 256, 64, 9, causal=False),
    Shape(1, 2, 1, 333, 700, 128, 100, 20, dtype=FP32),
    Shape(1, 1, 1, 200, 600, 256, 50, 150, dtype=FP32),
    Shape(1, 1, 1, 6000, 6000, 64, 100, 2),     # a sink's walk in many parts
    Shape(1, 2, 1, 5000, 5000, 256, 200, 260),
    # as many sinks as a narrow block holds, and one more or less, on single CTAs and on pairs
    *[Shape(1, Hq, 1, 300, 800, D, 150, S, dtype=t)
      for S, t in ((16, BF16), (17, BF16), (31, FP16), (32, BF16), (33, FP16))
      for Hq, D in ((1, 64), (1, 128), (2, 128), (2, 256))],
    # the last of several far blocks narrow, or not, with tiles that see the first of them far alone
    *[Shape(1, Hq, 1, 700, 700, D, 130, S, dtype=t)
      for S, t in ((129, BF16), (160, FP16), (161, BF16), (270, FP16))
      for Hq, D in ((1, 64), (1, 128), (2, 128), (1, 256), (2, 256))],
]


def inputs(sh, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(H, L):
        return torch.randn((sh.B, H, L, sh.D), generator=g, device="cuda").to(sh.dtype)

    x = {"q": normal(sh.Hq, sh.Lq), "k": normal(sh.Hkv, sh.Lk), "v": normal(sh.Hkv, sh.Lk),
         "do": normal(sh.Hq, sh.Lq) * 0.125}
    return x


def visible(sh):
    at = torch.arange(sh.Lq, device="cuda")[:, None] + sh.Lk - sh.Lq
    key = torch.arange(sh.Lk, device="cuda")
    d = at - key
    return (d >= (0 if sh.causal else 1 - sh.W)) & ((d < sh.W) | (key < sh.S))


def dense(sh, x):
    """o, lse, dq, dk, dv in 64 bits, from the formulas, a head at a time."""
    G, scale, see = sh.Hq // sh.Hkv, 1 / math.sqrt(sh.D), visible(sh)
    q, k, v, do = (x[n].double() for n in ("q", "k", "v", "do"))
    o, dq = torch.zeros_like(q), torch.zeros_like(q)
    dk, dv = torch.zeros_like(k), torch.zeros_like(v)
    lse = q.new_zeros(q.shape[:3])
    for b in range(sh.B):
        for h in range(sh.Hq):
            s = torch.where(see, q[b, h] @ k[b, h // G].T * scale, -math.inf)
            lse[b, h] = torch.logsumexp(s, -1)
            p = torch.exp(s - lse[b, h, :, None])
            o[b, h] = p @ v[b, h // G]
            dp = do[b, h] @ v[b, h // G].T
            ds = p * (dp - (do[b, h] * o[b, h]).sum(-1, keepdim=True)) * scale
            dq[b, h] = ds @ k[b, h // G]
            dk[b, h // G] += ds.T @ q[b, h]
            dv[b, h // G] += p.T @ do[b, h]
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def step(swa, sh, x, **kw):
    o, lse = swa.swa_attn_fwd(x["q"], x["k"], x["v"], sh.W, causal=sh.causal, sinks=sh.S)
    dq, dk, dv = swa.swa_attn_bwd(x["q"], x["k"], x["v"], o, x["do"], lse, sh.W, causal=sh.causal,
                                  sinks=sh.S, **kw)
    swa.swa_check_device()
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def near(got, ref, what):
    assert torch.isfinite(got).all(), what
    err, norm = (got.double() - ref).norm().item(), ref.norm().item()
    assert err <= REL * norm, f"{what}: {err / norm:.2e}"


@pytest.mark.parametrize("sh", SHAPES, ids=Shape.name)
def test_parity(swa, sh):
    x = inputs(sh)
    ref, got = dense(sh, x), step(swa, sh, x)
    assert (got["lse"].double() - ref["lse"]).abs().max().item() <= LSE
    S = min(sh.S, sh.Lk)
    for name in ("o", "dq", "dk", "dv"):
        assert got[name].dtype == sh.dtype and got[name].shape == x["q" if name in ("o", "dq") else "k"].shape
        near(got[name], ref[name], name)
        if name in ("dk", "dv"):
            near(got[name][:, :, :S], ref[name][:, :, :S], name + " of the sinks")
            hidden = ~visible(sh).any(0)
            assert not got[name][:, :, hidden].any(), name + " of keys that nobody sees"


def test_gradients_are_those_of_differences(swa):
    """dk along a random direction: the formula's against the difference of the dense loss in 64 bits,
    then the kernel's, whose error along a unit-normal direction is that of its norm times a normal
    number (4 of them allowed)."""
    sh = Shape(1, 2, 1, 260, 260, 64, 40, 3)
    x = inputs(sh)
    ref = dense(sh, x)
    eps, name = 1e-6, "k"
    g = torch.Generator(device="cuda").manual_seed(9)
    u = torch.randn(x[name].shape, generator=g, device="cuda", dtype=torch.float64)

    def loss(t):
        y = {k: v.double() for k, v in x.items()}
        y[name] = y[name] + t * u
        return (dense(sh, y)["o"] * x["do"].double()).sum()

    slope = ((loss(eps) - loss(-eps)) / (2 * eps)).item()
    assert abs(slope - (ref["dk"] * u).sum().item()) <= 1e-6 * max(1.0, abs(slope))
    got = step(swa, sh, x)
    assert abs((got["dk"].double() * u).sum().item() - slope) <= REL * ref["dk"].norm().item() * 4


@pytest.mark.parametrize("sh", [Shape(1, 4, 2, 500, 500, 128, 64, 0), Shape(1, 4, 2, 500, 500, 256, 64, 0),
                                Shape(1, 3, 1, 200, 500, 64, 500, 9), Shape(1, 2, 1, 300, 300, 128, 4000, 9)],
                         ids=Shape.name)
def test_without_sinks_or_with_a_wide_window_nothing_changes(swa, sh):
    x = inputs(sh)
    got = step(swa, sh, x)
    o, lse = swa.swa_attn_fwd(x["q"], x["k"], x["v"], sh.W)
    grads = swa.swa_attn_bwd(x["q"], x["k"], x["v"], o, x["do"], lse, sh.W)
    for a, b in zip(got.values(), (o, lse, *grads)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("D,Hq", [(64, 1), (128, 1), (128, 2), (256, 1), (256, 2)])
def test_neighbours_of_far_sinks_are_not_read(swa, D, Hq):
    """NaN between the sinks and the windows of the later queries reaches none of them."""
    sh = Shape(1, Hq, 1, 256, 900, D, 64, 5)  # windows begin at key 580
    x = inputs(sh)
    clean = step(swa, sh, x)
    y = dict(x)
    for n in ("k", "v"):
        y[n] = x[n].clone()
        y[n][:, :, 5:500] = math.nan
    got = step(swa, sh, y)
    for n in ("o", "lse", "dq"):
        assert torch.equal(got[n], clean[n]), n
    for n in ("dk", "dv"):
        assert torch.equal(got[n][:, :, :5], clean[n][:, :, :5]), n
        assert torch.equal(got[n][:, :, 512:], clean[n][:, :, 512:]), n


@pytest.mark.parametrize("sh", [Shape(2, 4, 2, 700, 700, 128, 64, 4), Shape(1, 2, 1, 700, 1300, 256, 64, 200)],
                         ids=Shape.name)
def test_same_bits_again_and_in_a_graph_on_other_data(swa, sh):
    x, y = inputs(sh, 1), inputs(sh, 2)
    want = step(swa, sh, y)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = step(swa, sh, y)
    torch.cuda.current_stream().wait_stream(s)
    for n in want:
        assert torch.equal(want[n], again[n]), n
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = swa.swa_attn_fwd(x["q"], x["k"], x["v"], sh.W, sinks=sh.S)
        grads = swa.swa_attn_bwd(x["q"], x["k"], x["v"], o, x["do"], lse, sh.W, sinks=sh.S)
    for n in x:
        x[n].copy_(y[n])
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    swa.swa_check_device()
    for n, t in zip(want, (o, lse, *grads)):
        assert torch.equal(want[n], t), n


def test_autograd_and_given_buffers(swa):
    sh = Shape(1, 4, 2, 300, 300, 128, 50, 6)
    x = inputs(sh)
    want = step(swa, sh, x)
    q, k, v = (x[n].clone().requires_grad_() for n in "qkv")
    o = swa.SlidingWindowAttention.apply(q, k, v, sh.W, None, True, sh.S)
    o.backward(x["do"])
    for n, t in (("o", o), ("dq", q.grad), ("dk", k.grad), ("dv", v.grad)):
        assert torch.equal(want[n], t.detach()), n
    need = swa.swa_attn_sinks_workspace_bytes(sh.B, sh.Hq, sh.Hkv, sh.Lq, sh.Lk, sh.D, sh.W, sh.S,
                                              backward=True)
    guard = torch.full((need + 256,), 7, dtype=torch.uint8, device="cuda")
    got = step(swa, sh, x, workspace=guard[:need])
    assert (guard[need:] == 7).all()
    for n in want:
        assert torch.equal(want[n], got[n]), n
    with pytest.raises(swa.SwaError, match="WORKSPACE"):
        step(swa, sh, x, workspace=guard[:need - 1])


def test_autograd_captured(swa):
    sh = Shape(1, 4, 2, 300, 300, 128, 64, 4)
    x, y = inputs(sh, 1), inputs(sh, 2)
    leaves = [x[n].clone().requires_grad_() for n in "qkv"]
    eager = swa.SlidingWindowAttention.apply(*leaves, sh.W, None, True, sh.S)
    eager.backward(x["do"])
    del eager  # a graph made outside the capture must not live on
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = swa.SlidingWindowAttention.apply(*leaves, sh.W, None, True, sh.S)
        grads = torch.autograd.grad(o, leaves, x["do"])
    with torch.no_grad():
        for t, n in zip(leaves, "qkv"):
            t.copy_(y[n])
    x["do"].copy_(y["do"])
    graph.replay()
    want = step(swa, sh, y)
    assert torch.equal(o, want["o"])
    for a, n in zip(grads, ("dq", "dk", "dv")):
        assert torch.equal(a, want[n]), n
