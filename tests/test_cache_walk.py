"""CPU checks of the cache attention with sinks: its walk against brute force, and what it refuses."""
import os
import shutil
import subprocess

import pytest

import sliding_window_flash_gb300 as swa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sliding_window_flash_gb300", "csrc")


def _run(tmp_path, header_dir):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("needs a host C++ compiler")
    exe = str(tmp_path / "cache_walk_check")
    subprocess.run([cxx, "-std=c++17", "-O2", f"-I{header_dir}",
                    os.path.join(ROOT, "tests", "cache_walk_check.cpp"), "-o", exe], check=True)
    return subprocess.run([exe], capture_output=True, text=True, timeout=120)


def test_walk_matches_brute_force(tmp_path):
    r = _run(tmp_path, CSRC)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout + r.stderr


@pytest.mark.parametrize("old,new", [
    ("far = (stop < first ? stop : first) - base;", "far = stop - base;"),
    ("first = wide > base ? wide : base;", "first = wide;"),
    ("i < far ? far0 + i : first + (i - far)", "i < far ? i : first + (i - far)"),
    ("count = n > 0 && end > r.base ?", "count = n > 0 ?"),
])
def test_the_check_rejects_planted_mistakes(tmp_path, old, new):
    src = open(os.path.join(CSRC, "swa_cache_split.h")).read()
    assert src.count(old) == 1, old
    (tmp_path / "swa_cache_split.h").write_text(src.replace(old, new))
    r = _run(tmp_path, tmp_path)
    assert r.returncode == 1 and r.stdout.startswith("failed"), r.stdout


def test_workspace_sizes():
    size = swa.swa_cache_attn_workspace_bytes
    args = (3, 8, 2, 2, 128, 500, 64)
    wide = size(*args, accumulate=True)
    assert size(*args, window=100, sinks=0, accumulate=True) == size(*args, window=100, accumulate=True)
    assert size(*args, window=100, sinks=4) == size(*args, window=100)
    assert size(*args, window=100, sinks=20000, accumulate=True) > size(*args, window=100, accumulate=True)
    assert size(*args, window=100, sinks=2**40, accumulate=True) <= wide
    assert size(*args, window=2**40, sinks=9, accumulate=True) == wide
    assert size(*args, window=100, sinks=-1) == 0


def test_shared_workspaces_and_refusals():
    size = swa.swa_cache_attn_workspace_bytes
    args = (3, 8, 2, 2, 128, 500, 64)
    assert size(*args, shared=100) > size(*args)
    assert size(*args, window=100, shared=0) == size(*args, window=100)
    assert size(1, *args[1:], shared=100) == size(1, *args[1:])     # nobody to share with
    assert size(*args, shared=501) == 0 and size(*args, shared=-1) == 0
    assert size(*args, shared=1, accumulate=True) == 0
    assert size(2, 2, 1, 64, 64, 8, 64, shared=1) > 0
    assert size(2, 2050, 1, 64, 64, 8, 64, shared=1) == 0           # too many rows to a kv head


def call(**kw):
    from sliding_window_flash_gb300.cache import _CCache
    a = dict(B=2, Hq=2, Hkv=1, T=1, window=10, sinks=0, shared=1, scale=0.1, acc=0, dtype=0, max_pages=4,
             size=1 << 30)
    a.update(kw)
    c = _CCache(16, 16, 16, 16, 16, 8, a["Hkv"], 32, 64)
    return swa.load().swa_cache_attn_shared(c, 16, a["max_pages"], 16, None, 16, 16, 16, a["B"], a["Hq"],
                                            a["T"], a["window"], a["sinks"], a["shared"], a["scale"],
                                            a["acc"], a["dtype"], 16, a["size"], None)


@pytest.mark.parametrize("kw,code", [(dict(shared=-1), 1), (dict(shared=5), 1), (dict(acc=1), 1),
                                     (dict(sinks=-1), 1), (dict(sinks=-1, shared=0), 1),
                                     (dict(Hq=1025, T=64), 1), (dict(size=100), 6)], ids=str)
def test_bad_arguments(kw, code):
    assert call(**kw) == code
