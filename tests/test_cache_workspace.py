"""The attention's workspace under a window: how many chunks a call can see, by brute force; its size; and
an accumulating call in exactly that many bytes."""
import os
import shutil
import subprocess

import pytest
import torch

import sliding_window_flash_gb300 as swa_mod

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sliding_window_flash_gb300", "csrc")


def _run(tmp_path, header_dir):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("needs a host C++ compiler")
    exe = str(tmp_path / "check")
    subprocess.run([cxx, "-std=c++17", "-O2", f"-I{header_dir}",
                    os.path.join(ROOT, "tests", "cache_chunks_check.cpp"), "-o", exe],
                   check=True, capture_output=True, text=True)
    return subprocess.run([exe], capture_output=True, text=True, timeout=120)


def test_most_chunks_matches_brute_force(tmp_path):
    r = _run(tmp_path, CSRC)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout + r.stderr


@pytest.mark.parametrize("old,new", [
    ("static_cast<int64_t>(window) + T - 1;", "static_cast<int64_t>(window) + T - 2;"),
    ("+ ck - 2) / ck + 1;", "+ ck - 1) / ck;"),
    ("+ ck - 2) / ck + 1;", "+ ck) / ck + 1;"),
    ("span < slots ? span : slots", "span"),
    ("span < slots ? span : slots", "span < slots ? slots : span"),
])
def test_most_chunks_check_rejects_planted_mistakes(tmp_path, old, new):
    src = open(os.path.join(CSRC, "swa_cache_split.h")).read()
    assert src.count(old) == 1, old
    hdr = tmp_path / "hdr"
    hdr.mkdir()
    (hdr / "swa_cache_split.h").write_text(src.replace(old, new))
    r = _run(tmp_path, str(hdr))
    assert r.returncode == 1 and r.stdout.startswith("failed"), r.stdout


# ---- sizes -------------------------------------------------------------------------------------

@pytest.fixture(scope="module")
def lib():
    from sliding_window_flash_gb300 import build

    if not os.path.exists(swa_mod.library_path()):
        build.build()
    return swa_mod.load()


SIZES = [  # B, Hq, H, T, D, page
    (64, 32, 8, 1, 128, 64), (1, 32, 16, 1, 128, 64), (8, 32, 4, 5, 64, 32), (12, 32, 16, 5, 256, 32),
    (4, 64, 4, 64, 128, 128), (2000, 8, 2, 1, 128, 64),
]


@pytest.mark.parametrize("B,Hq,H,T,D,page", SIZES)
def test_windowed_size_does_not_follow_the_table(lib, B, Hq, H, T, D, page):
    size, any_window = lib.swa_cache_attn_window_workspace_bytes, lib.swa_cache_attn_workspace_bytes
    for window in (1, 100, 1024):
        assert size(B, Hq, H, T, D, 1 << 16, page, window, 1) == size(B, Hq, H, T, D, 1 << 13, page,
                                                                     window, 1)
    ck, R = 16 if D == 256 else 32, Hq // H * T
    tile = 16 if R <= 16 else 32 if R <= 32 else 64
    rows = -(-R // tile) * min(R, tile)
    base = size(B, Hq, H, T, D, 4096, page, 1, 0)
    for width in (1, 3, 64, 4096):
        slots = width * page
        whole = any_window(B, Hq, H, T, D, width, page, 1)
        assert any_window(B, Hq, H, T, D, width, page, 0) == base  # without scores: one size
        assert whole - base <= min(B, 1024) * H * rows * slots * 4 + 512
        last = 0
        for window in (1, 2, 31, 32, 33, 1000, 5000, slots - 1, slots, slots + 1, 2**31 - 1):
            if window < 1:
                continue
            got = size(B, Hq, H, T, D, width, page, window, 1)
            most = min(slots // ck, (min(window + T - 1, slots) + ck - 2) // ck + 1)
            need = min(B, 1024) * H * rows * most * ck * 4
            assert base + need - 256 <= got <= min(whole, base + need + (2 << 20) + 256)
            assert window < last or got >= size(B, Hq, H, T, D, width, page, max(last, 1), 1)
            last = window
        assert size(B, Hq, H, T, D, width, page, slots, 1) == whole


def test_windowed_size_of_refused_calls_is_zero(lib):
    size = lib.swa_cache_attn_window_workspace_bytes
    good = (2, 4, 2, 1, 128, 4, 64, 9, 1)
    assert size(*good) > 0
    for at, value in ((0, 0), (1, 3), (2, 0), (3, 0), (3, 65), (4, 96), (5, 0), (5, 1 << 24), (6, 48),
                      (7, 0), (7, -5)):
        assert size(*good[:at], value, *good[at + 1:]) == 0


def test_a_window_takes_megabytes_of_a_long_table(lib):
    """64 sequences, 32 / 8 heads, tables of 131,072 slots, a window of 1024."""
    public = swa_mod.swa_cache_attn_workspace_bytes
    sizes = (64, 32, 8, 1, 128, 2048, 64, True)
    assert public(*sizes) > 1 << 30
    assert public(*sizes, window=1024) < 16 << 20
    assert public(*sizes, window=2**40) == public(*sizes) and public(*sizes, window=-2**32 + 9) == 0


# ---- on the GPU --------------------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("B,H_q,H,D,page,T,window,dtype", [
    # the scores fill their whole units of 2 MB, every sequence has the most chunks that it can have
    (64, 32, 8, 64, 64, 1, 225, torch.bfloat16),
    (64, 32, 8, 128, 32, 1, 225, torch.float16),
    (16, 64, 4, 64, 64, 8, 218, torch.bfloat16),
    (32, 32, 8, 256, 32, 2, 240, torch.bfloat16),
])
def test_accumulation_in_the_windows_bytes(swa, B, H_q, H, D, page, T, window, dtype):
    """Exactly the bytes of the window's size, guarded on both sides, under a table far wider than it."""
    import cache_ref as ref
    from test_cache import _cache, _gen, _ints, _near, _table

    g = _gen(D + T)
    ck = 16 if D == 256 else 32
    lens = [window - 1 + ck - 1 + ck * (b % 5) for b in range(B)]
    width = -(-(max(lens) + T) // page)
    cache = _cache(swa, g, B * width, H, D, page, spread=3)
    wide = torch.full((B, 65536 // page), -1, dtype=torch.int32, device="cuda")
    wide[:, :width] = table = _table(g, B, width)
    q = torch.randn((B, H_q, T, D), generator=g, device="cuda").to(dtype)
    pool = ref.pool_of(cache)
    o, lse, to, tl, tw = ref.attn(pool, table, lens, q, window, accumulate=True)
    need = swa.swa_cache_attn_workspace_bytes(B, H_q, H, T, D, wide.shape[1], page, True, window=window)
    assert need < swa.swa_cache_attn_workspace_bytes(B, H_q, H, T, D, wide.shape[1], page, True)
    held = torch.full((need + 2 * 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    with pytest.raises(swa.SwaError, match="WORKSPACE"):
        swa.swa_cache_attn(q, cache, wide, _ints(lens), window, accumulate=True,
                           workspace=held[4096:4096 + need - 16])
    go, gl = swa.swa_cache_attn(q, cache, wide, _ints(lens), window, accumulate=True,
                                workspace=held[4096:4096 + need])
    swa.swa_check_device()
    _near(go, o, to, "o")
    _near(gl, lse, tl, "lse")
    _near(cache.weight, pool["weight"], tw, "weight")
    assert (held[:4096] == 0xA5).all() and (held[-4096:] == 0xA5).all()


@pytest.mark.gpu
def test_a_windowed_call_allocates_for_its_window(swa):
    """64 sequences under tables of 131,072 slots: the call's own workspace is the window's."""
    B, H_q, H, D, page, window = 64, 32, 8, 128, 64, 1024
    cache = swa.SwaCache.empty(32, H, D, page)
    table = torch.zeros((B, 131072 // page), dtype=torch.int32, device="cuda")
    table[:, 0] = torch.arange(B, device="cuda") % 32
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    q = torch.randn((B, H_q, 1, D), device="cuda").bfloat16()
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    swa.swa_cache_attn(q[:32], cache, table[:32], lens[:32], window, accumulate=True)
    swa.swa_check_device()
    assert torch.cuda.max_memory_allocated() - before < 64 << 20
