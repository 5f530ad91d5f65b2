"""The training calls refuse workspaces whose bytes are not all on the tensors' GPU: shown on the CPU,
with the library replaced by a recorder."""
import pytest
import torch

import sliding_window_flash_gb300 as swa


class Library:
    """Every size is 4096 bytes, every call succeeds and is noted."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return lambda *a: 4096

        def call(*a):
            self.calls.append((name, a))
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    lib = Library()
    monkeypatch.setattr(swa, "load", lambda: lib)
    monkeypatch.setattr(swa, "_check_tensor", lambda *a: None)
    monkeypatch.setattr(swa, "_stream_handle", lambda device: 0)
    return lib


def _tensors(dtype):
    q = torch.zeros((1, 2, 8, 64), dtype=dtype)
    k = torch.zeros((1, 1, 8, 64), dtype=dtype)
    return q, k, torch.zeros((1, 2, 8))


def _fwd_f32(ws):
    q, k, _ = _tensors(torch.float32)
    swa.swa_attn_fwd(q, k, k, 4, workspace=ws)


def _bwd(dtype, **kw):
    def run(ws):
        q, k, lse = _tensors(dtype)
        swa.swa_attn_bwd(q, k, k, q, q, lse, 4, workspace=ws, **kw)
    return run


def _phases(ws):
    q, k, lse = _tensors(torch.bfloat16)
    swa.swa_attn_bwd_phases(q, k, k, q, q, lse, 4, fused=True, workspace=ws)


CALLS = [_fwd_f32, _bwd(torch.float32), _bwd(torch.bfloat16), _bwd(torch.float16, fused=True),
         _bwd(torch.bfloat16, causal=False), _phases]


def _bad():
    u8 = torch.uint8
    return (torch.empty(1, dtype=u8).expand(1 << 20), torch.empty((64, 64), dtype=u8).t(),
            torch.empty(8192, dtype=u8, device="meta"), bytearray(8192))


@pytest.mark.parametrize("call", CALLS, ids=["fwd_f32", "bwd_f32", "bwd", "bwd_fused", "bwd_ex", "phases"])
def test_workspace_is_a_whole_tensor_on_the_gpu(lib, call):
    for bad in _bad():
        with pytest.raises((TypeError, ValueError), match="workspace"):
            call(bad)
    assert lib.calls == []
    good = torch.empty((2, 4096), dtype=torch.int16)
    call(good)
    used = [a for _, a in lib.calls if good.data_ptr() in a]
    assert used and all(a[a.index(good.data_ptr()) + 1] == 16384 for a in used)


@pytest.mark.parametrize("device", [None, "cuda", "cuda:0", 0, torch.device("cuda")])
def test_host_pipeline_workspace(lib, monkeypatch, device):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    q, k, lse = _tensors(torch.bfloat16)
    outs = (q, lse, q, k, k)
    for bad in _bad() + (torch.empty(8192, dtype=torch.uint8),):
        with pytest.raises((TypeError, ValueError), match="workspace"):
            swa.swa_attn_fwd_bwd_host(q, k, k, q, 4, outs=outs, workspace=bad, device=device)
    assert lib.calls == []


@pytest.mark.parametrize("device", ["cpu", torch.device("cpu"), "meta"])
def test_host_pipeline_runs_on_a_gpu_only(lib, monkeypatch, device):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    q, k, lse = _tensors(torch.bfloat16)
    with pytest.raises(ValueError, match="device"):
        swa.swa_attn_fwd_bwd_host(q, k, k, q, 4, outs=(q, lse, q, k, k), device=device)
    assert lib.calls == []


@pytest.mark.gpu
@pytest.mark.parametrize("device", [None, "cuda", 0])
def test_host_pipeline_takes_its_gpus_workspace(swa, device):
    g = torch.Generator().manual_seed(3)
    q, do = (torch.randn((1, 2, 256, 64), generator=g).bfloat16() for _ in range(2))
    k, v = (torch.randn((1, 1, 256, 64), generator=g).bfloat16() for _ in range(2))
    n = swa.swa_attn_host_workspace_bytes(1, 2, 1, 256, 64, 1)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    got = swa.swa_attn_fwd_bwd_host(q, k, v, do, 64, units_per_chunk=1, workspace=ws, device=device)
    torch.cuda.synchronize()
    want = swa.swa_attn_fwd_bwd_host(q, k, v, do, 64, units_per_chunk=1)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
