"""Calls one directly behind the other, without a kernel of torch's between them, and the early kernels that
test_early_launch.py does not reach: CTA pairs (an even group), D = 256 without them, fp32.  Each run is
compared, bit for bit, with one that waits for the GPU between all steps."""
import pytest
import torch

from test_cache_shared import setup
from test_cache_sinks import ints
from test_early_launch import serving, training

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
PAIR128, PAIR128_2, ODD256 = (1, 4, 2, 300, 128), (2, 4, 2, 700, 128), (1, 3, 1, 300, 256)
PAIR256, SINGLE64 = (1, 4, 2, 300, 256), (1, 3, 1, 300, 64)


def ways(swa, make):
    """What make(settle)() gives when it waits between all steps, then eager, on another stream and captured."""
    want = [t.clone() for t in make(torch.cuda.synchronize)()]
    torch.cuda.synchronize()

    def same(got, how):
        torch.cuda.synchronize()
        swa.swa_check_device()
        for i, (a, b) in enumerate(zip(want, got)):
            assert torch.equal(a, b), f"{how}: output {i}"

    same(make(lambda: None)(), "eager")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = make(lambda: None)()
    torch.cuda.current_stream().wait_stream(side)
    same(got, "another stream")
    run = make(lambda: None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    graph.replay()
    same(got, "captured")


@pytest.mark.parametrize("sizes", [PAIR128, PAIR128_2, ODD256, PAIR256], ids=str)
@pytest.mark.parametrize("make", [training, serving])
def test_nothing_overtakes(swa, make, sizes):
    ways(swa, lambda settle: make(swa, sizes, settle))


@pytest.mark.parametrize("sizes", [PAIR128, ODD256, SINGLE64], ids=str)
def test_two_streams_at_once(swa, sizes):
    makes = (training, serving)
    wants = [[t.clone() for t in make(swa, sizes, torch.cuda.synchronize)()] for make in makes]
    streams = [torch.cuda.Stream() for _ in makes]
    torch.cuda.synchronize()
    gots = [[], []]
    for _ in range(6):
        for make, stream, got in zip(makes, streams, gots):
            with torch.cuda.stream(stream):
                got.append(make(swa, sizes, lambda: None)())
    torch.cuda.synchronize()
    swa.swa_check_device()
    for want, runs in zip(wants, gots):
        for got in runs:
            assert all(torch.equal(a, b) for a, b in zip(want, got))


class Layer:
    """A layer with its inputs and buffers, and its backward as a call that makes nothing."""

    def __init__(self, swa, sizes, dtype, seed, workspace=None):
        B, Hq, H, N, D = sizes
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.swa, self.kw = swa, dict(window=40, sinks=3)
        self.q, self.do = (torch.randn((B, Hq, N, D), generator=g, device="cuda").to(dtype) for _ in range(2))
        self.k, self.v = (torch.randn((B, H, N, D), generator=g, device="cuda").to(dtype) for _ in range(2))
        need = swa.swa_attn_sinks_workspace_bytes(B, Hq, H, N, N, D, 40, 3, dtype=dtype, backward=True)
        self.need, self.workspace = need, workspace
        self.o, self.lse = torch.empty_like(self.q), torch.empty((B, Hq, N), device="cuda")
        self.grads = [torch.empty_like(x) for x in (self.q, self.k, self.v)]

    def forward(self):
        self.swa.swa_attn_fwd(self.q, self.k, self.v, out=self.o, lse=self.lse, workspace=self.workspace, **self.kw)

    def backward(self):
        dq, dk, dv = self.grads
        self.swa.swa_attn_bwd(self.q, self.k, self.v, self.o, self.do, self.lse, dq=dq, dk=dk, dv=dv,
                              workspace=self.workspace, **self.kw)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("sizes", [SINGLE64, PAIR128, (1, 3, 1, 300, 128), PAIR256, ODD256], ids=str)
def test_layers_on_one_workspace(swa, sizes, dtype):
    """Forwards and backwards of layers large and small in turn, all over one workspace: what a kernel keeps
    at its start of the layer before must not reach the next one's results."""
    B, Hq, H, N, D = sizes
    layers = [Layer(swa, (4, Hq, H, 3000, D), dtype, 1)] + [Layer(swa, sizes, dtype, s) for s in (2, 3, 4)]
    space = torch.zeros(max(y.need for y in layers), dtype=torch.uint8, device="cuda")
    for y in layers:
        y.workspace = space

    def make(settle):
        def run():
            out = []
            for y in layers + layers[::-1] + [layers[0], layers[2]]:
                y.forward()
                settle()
                y.backward()
                settle()
                out.append(y)
            return [t for y in layers for t in (y.o, y.lse, *y.grads)]
        return run

    ways(swa, make)


@pytest.mark.parametrize("D,page,window,sinks,shared", [(64, 32, 700, 2, 20), (128, 64, 1 << 20, 0, 20),
                                                         (256, 32, 300, 4, 30)])
def test_answers_as_the_next_queries(swa, D, page, window, sinks, shared):
    """Each call's queries are what the call directly ahead of it has written, over them."""
    B, Hq, H, T = 6, 4, 2, 2
    cache, table, g = setup(swa, 12, B, H, D, page, shared, shared + 2)
    lens = ints([shared * page + 5 * b - 100 * (b == 2) for b in range(B)])
    first = torch.randn((B, Hq, T, D), generator=g, device="cuda").bfloat16()
    lse = torch.empty((B, Hq, T), device="cuda")

    def make(settle):
        space = torch.empty(max(swa.swa_cache_attn_workspace_bytes(B, Hq, H, T, D, shared + 2, page, window=window,
                                                                   sinks=sinks, shared=n)
                                for n in (0, shared)), dtype=torch.uint8, device="cuda")
        x = first.clone()

        def run():
            x.copy_(first)
            settle()
            for i in range(12):
                swa.swa_cache_attn(x, cache, table, lens, window, scale=1.0, out=x, lse=lse, workspace=space,
                                   sinks=sinks, shared=shared if i % 3 else 0)
                settle()
            return x, lse
        return run

    ways(swa, make)
