"""What the cache calls refuse before anything is launched, shown on the CPU (the launch is replaced by
a recorder), and the same refusals on the GPU."""
import ctypes

import pytest
import torch

import sliding_window_flash_gb300 as swa
from sliding_window_flash_gb300 import cache as mod

CPU = torch.device("cpu")


@pytest.fixture
def calls(monkeypatch):
    """Calls take CPU tensors for GPU ones and are recorded instead of launched."""
    seen = []
    monkeypatch.setattr(mod, "_check", lambda *a, **k: None)
    monkeypatch.setattr(mod, "_good", lambda *a, **k: True)
    monkeypatch.setattr(mod, "_run", lambda name, index, *args: seen.append((name, args)))
    monkeypatch.setattr(mod, "_attn_space", lambda *a: 4096)
    monkeypatch.setattr(mod, "_weights_space", lambda *a: 4096)
    return seen


def _cpu_cache(pages=4, H=2, page=32, D=64):
    k = torch.zeros((pages, H, page, D), dtype=torch.uint8).view(torch.float8_e4m3fn)
    s, w = torch.ones((pages, H)), torch.zeros((pages, H, page))
    c = object.__new__(swa.SwaCache)
    mod._put(c, "held", (k, k, s, s, w, CPU, tuple(k.shape)))
    return c


def _attn(**kw):
    q = torch.zeros((1, 4, 1, 64), dtype=torch.bfloat16)
    table, lens = torch.zeros((1, 4), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    return swa.swa_cache_attn(q, _cpu_cache(), table, lens, kw.pop("window", 9), **kw)


def _weights(**kw):
    q = torch.zeros((1, 4, 8, 64), dtype=torch.bfloat16)
    return swa.swa_attn_key_weights(q, q[:, :2], torch.zeros((1, 4, 8)), kw.pop("window", 9), **kw)


# ---- workspaces --------------------------------------------------------------------------------

@pytest.mark.parametrize("call", [_attn, _weights], ids=["attn", "weights"])
def test_workspace_is_a_whole_tensor_on_the_gpu(calls, call):
    """An expanded tensor holds less than its shape says; another device's memory is not the kernels'."""
    u8 = torch.uint8
    for bad in (torch.empty(1, dtype=u8).expand(1 << 20), torch.empty((64, 64), dtype=u8).t(),
                torch.empty(8192, dtype=u8)[::2], torch.empty(8192, dtype=u8, device="meta"),
                bytearray(8192), 8192):
        with pytest.raises((TypeError, ValueError), match="workspace"):
            call(workspace=bad)
    assert calls == []
    good = torch.empty((4, 4096), dtype=torch.int16)
    call(workspace=good)
    call()
    (_, given), (_, own) = calls
    assert (good.data_ptr(), 32768) == tuple(a for a in given if a in (good.data_ptr(), 32768))
    assert 4096 in own


@pytest.mark.gpu
def test_workspace_refusals_on_the_gpu(swa):
    cache = swa.SwaCache.empty(4, 2, 64, page=32)
    q = torch.zeros((1, 4, 1, 64), dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((1, 2, 8, 64), dtype=torch.bfloat16, device="cuda")
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    lse = torch.zeros((1, 4, 8), device="cuda")
    n = 1 << 26
    wrong = (torch.empty(n, dtype=torch.uint8), torch.empty(1, dtype=torch.uint8, device="cuda").expand(n))
    for bad in wrong:
        with pytest.raises(ValueError, match="workspace"):
            swa.swa_cache_attn(q, cache, table, lens, 9, workspace=bad)
        with pytest.raises(ValueError, match="workspace"):
            swa.swa_attn_key_weights(q.expand(1, 4, 8, 64).contiguous(), k, lse, 9, workspace=bad)
    fine = torch.empty((2, n // 2), dtype=torch.uint8, device="cuda")
    swa.swa_cache_attn(q, cache, table, lens, 9, workspace=fine)
    swa.swa_attn_key_weights(q.expand(1, 4, 8, 64).contiguous(), k, lse, 9, workspace=fine)
    swa.swa_check_device()


# ---- numbers that a C int does not hold --------------------------------------------------------

def _passed(calls, value_at):
    """What the last call's C function sees of argument `value_at`."""
    return ctypes.c_int(calls[-1][1][value_at]).value


@pytest.mark.parametrize("window", [2**32 + 5, 2**31, 2**40, 10**30])
def test_windows_past_an_int_see_everything(calls, window):
    _attn(window=window)
    assert _passed(calls, 11) == 2**31 - 1
    _weights(window=window)
    assert _passed(calls, 10) == 2**31 - 1


@pytest.mark.parametrize("window", [-2**32 + 5, -2**31 - 1, -10**30, 0, -1])
def test_windows_below_one_stay_below_one(calls, window):
    _attn(window=window)
    assert _passed(calls, 11) < 1
    _weights(window=window)
    assert _passed(calls, 10) < 1


def _evict(budget, recent):
    table, lens = torch.zeros((1, 4), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    return swa.swa_cache_evict(_cpu_cache(), table, lens, torch.zeros((1, 2), dtype=torch.int32), budget,
                               recent)


def test_evict_numbers_past_an_int(calls):
    for recent in (2**32, 2**32 + 3, 2**31, 10**30):
        _evict(20, recent)
        assert _passed(calls, 6) == 20 and _passed(calls, 7) > 20
    for recent in (-2**32, -2**32 + 3, -2**31 - 1, -1):
        _evict(20, recent)
        assert _passed(calls, 7) < 0
    _evict(20, 3)
    assert _passed(calls, 7) == 3
    done = len(calls)
    for budget in (2**32 + 20, 2**31, 2**30, -2**32 + 20, 0):
        with pytest.raises(ValueError, match="budget"):
            _evict(budget, 3)
    assert len(calls) == done


# ---- a workspace's size belongs to a GPU -------------------------------------------------------

def test_workspace_sizes_are_the_tensors_gpus(calls, monkeypatch):
    """GPUs may differ in SMs: a size is asked for with the tensors' GPU current, and not handed on."""
    monkeypatch.undo()
    assert mod._t.f32 is torch.float32  # the names are loaded
    now, seen = [0], []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.was, now[0] = now[0], self.index

        def __exit__(self, *_):
            now[0] = self.was

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(mod._t, "current_device", lambda: now[0])
    monkeypatch.setattr(mod, "_check", lambda *a, **k: None)
    monkeypatch.setattr(mod, "_good", lambda *a, **k: True)
    monkeypatch.setattr(mod, "_run", lambda name, index, *args: seen.append(args))
    for name in filter(lambda n: n.endswith("workspace_bytes"), mod.SIGNATURES):
        monkeypatch.setitem(mod._entries, name, lambda *sizes: 1000 + now[0] + sizes[0])
    sizes = getattr(mod._attn_space, "cache_clear", None), getattr(mod._weights_space, "cache_clear", None)
    try:
        for index in (0, 3, 0, 5):
            monkeypatch.setattr(mod, "_tables", lambda *a: (1, 4, index))
            _attn()
            assert seen[-1][-1] == 1001 + index and now[0] == 0
        now[0] = 5
        _attn()
        assert seen[-1][-1] == 1006
        monkeypatch.setattr(mod, "_tables", lambda *a: (1, 4, 0))
        _attn()
        assert seen[-1][-1] == 1001 and now[0] == 5
        assert mod._weights_space(3, 1, 4) == 1004 and mod._weights_space(5, 1, 4) == 1006
        assert now[0] == 5
        # the public forms answer for the current GPU
        assert swa.swa_cache_attn_workspace_bytes(1, 4, 2, 1, 64, 4, 32) == 1006
        now[0] = 2
        assert swa.swa_cache_attn_workspace_bytes(1, 4, 2, 1, 64, 4, 32) == 1003
        assert swa.swa_attn_key_weights_workspace_bytes(1, 4, 2, 8, 8, 64, 4) == 1003
    finally:
        for clear in filter(None, sizes):
            clear()


# ---- sizes that the call refuses ---------------------------------------------------------------

@pytest.fixture(scope="module")
def lib():
    import os

    from sliding_window_flash_gb300 import build

    if not os.path.exists(swa.library_path()):
        build.build()
    return swa.load()


@pytest.mark.parametrize("sizes", [
    (1, 2**31 - 1, 1, 64, 64, 4, 64), (1, 2**31 - 1, 1, 2, 64, 4, 64), (65536, 4, 2, 1, 64, 4, 64),
    (2**31 - 1, 2**31 - 1, 2**31 - 1, 1, 64, 4, 64), (1, 70000, 70000, 1, 64, 4, 64),
    (40000, 60000, 60000, 1, 64, 4, 64), (65535, 64, 1, 512, 64, 4, 64), (1000, 40000, 4, 64, 64, 4, 64),
])
def test_size_of_refused_calls_is_zero(lib, sizes):
    for acc in (0, 1):
        assert lib.swa_cache_attn_workspace_bytes(*sizes, acc) == 0
    largest = lib.swa_cache_attn_workspace_bytes(1024, 65535, 1, 31, 64, 2**24 - 1, 32, 1)
    assert 0 < largest < 2**63  # counted without wrapping
