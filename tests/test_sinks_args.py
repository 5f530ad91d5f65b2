"""What the calls with sinks refuse, and the walk over key blocks that their kernels share: on the CPU."""
import os
import shutil
import subprocess

import pytest
import torch

import sliding_window_flash_gb300 as swa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sliding_window_flash_gb300", "csrc")
INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 1, 2, 3, 6


def fwd(B=1, Hq=2, Hkv=1, Lq=64, Lk=64, D=64, W=16, S=4, causal=1, scale=0.125, dtype=0, ptr=16, ws=None,
        size=0):
    return swa.load().swa_attn_fwd_sinks(ptr, ptr, ptr, ptr, ptr, B, Hq, Hkv, Lq, Lk, D, W, S, causal,
                                         scale, dtype, ws, size, None)


def bwd(B=1, Hq=2, Hkv=1, Lq=64, Lk=64, D=64, W=16, S=4, causal=1, scale=0.125, dtype=0, ptr=16, ws=4096,
        size=1 << 30):
    return swa.load().swa_attn_bwd_sinks(*[ptr] * 9, B, Hq, Hkv, Lq, Lk, D, W, S, causal, scale, dtype, ws,
                                         size, None)


BAD = [(dict(S=-1), INVALID), (dict(dtype=3), INVALID), (dict(dtype=-1), INVALID), (dict(ptr=None), INVALID),
       (dict(causal=2), INVALID), (dict(W=0), INVALID), (dict(Lq=65), INVALID), (dict(Hq=3, Hkv=2), INVALID),
       (dict(scale=float("nan")), INVALID), (dict(scale=0.0), INVALID), (dict(B=0), INVALID),
       (dict(D=96), UNSUPPORTED), (dict(ptr=8), MISALIGNED)]


@pytest.mark.parametrize("call", [fwd, bwd])
@pytest.mark.parametrize("kw,code", BAD, ids=str)
def test_bad_arguments(call, kw, code):
    assert call(**kw) == code


def test_workspaces():
    assert bwd(ws=None) == WORKSPACE and bwd(size=100) == WORKSPACE
    assert fwd(dtype=2) == WORKSPACE and bwd(dtype=2, size=1000) == WORKSPACE
    size = swa.swa_attn_sinks_workspace_bytes
    args = (1, 2, 1, 64, 64, 64, 16)
    assert size(*args, 4) == 0
    base = swa.swa_attn_bwd_workspace_bytes(1, 2, 64, 64)
    part = size(*args, 4, backward=True) - base
    assert part > 0 and part % (2 * 4 * 64 * 4) == 0          # whole parts of dK and dV rows
    assert size(*args, 0, backward=True) == base
    assert size(1, 2, 1, 64, 64, 64, 64, 4, backward=True) == base  # the window hides nothing
    f32 = swa.swa_attn_f32_workspace_bytes(1, 2, 1, 64, 64, 64)
    assert size(*args, 4, dtype=torch.float32) == f32
    assert size(*args, 4, dtype=torch.float32, backward=True) == f32 + part
    assert size(0, *args[1:], 4, backward=True) == 0
    assert size(*args, 2**40, backward=True) == size(*args, 64, backward=True)  # more than an int holds
    raw = swa.load().swa_attn_sinks_workspace_bytes
    assert raw(*args, 4, 1, 0, 2) == 0 and raw(*args, 4, 2, 0, 1) == 0 and raw(*args, 4, 1, 5, 1) == 0
    assert raw(*args, -1, 1, 0, 1) == 0


def test_binding():
    q, k = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16), torch.zeros(1, 1, 8, 64, dtype=torch.bfloat16)
    for bad in (-1, -2**40):
        with pytest.raises(ValueError, match="negative"):
            swa.swa_attn_fwd(q, k, k, 4, sinks=bad)
        with pytest.raises(ValueError, match="negative"):
            swa.swa_attn_bwd(q, k, k, q, q, q, 4, sinks=bad)
        with pytest.raises(ValueError, match="negative"):
            swa.swa_attn_sinks_workspace_bytes(1, 2, 1, 8, 8, 64, 4, bad)
    with pytest.raises(ValueError, match="fused"):
        swa.swa_attn_bwd(q, k, k, q, q, q, 4, sinks=1, fused=True)
    with pytest.raises(ValueError, match="CUDA"):
        swa.swa_attn_fwd(q, k, k, 4, sinks=1)


def test_tensors_of_two_gpus_are_refused(monkeypatch):
    monkeypatch.setattr(swa, "_check_tensor", lambda *a: None)
    q, k = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16), torch.zeros(1, 1, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="expected cpu"):
        swa.swa_attn_fwd(q, k, k.to("meta"), 4, sinks=1)


def check(tmp_path, headers):
    cxx, cuda = shutil.which("g++") or shutil.which("c++"), os.path.join(
        os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    if cxx is None or not os.path.exists(os.path.join(cuda, "cuda_runtime.h")):
        pytest.skip("needs a host C++ compiler and the CUDA headers")
    exe = str(tmp_path / "sinks_check")
    subprocess.run([cxx, "-std=c++17", "-O2", f"-I{headers}", f"-I{cuda}",
                    os.path.join(ROOT, "tests", "sinks_check.cpp"), "-o", exe], check=True)
    return subprocess.run([exe], capture_output=True, text=True, timeout=300)


def test_key_walk(tmp_path):
    """The blocks of every query tile: each that holds a visible key, once, in order, far ones first."""
    r = check(tmp_path, CSRC)
    assert r.returncode == 0 and r.stdout.startswith("ok "), r.stdout + r.stderr


@pytest.mark.parametrize("old,new", [
    ("if (far > kb_lo) far = kb_lo;", "if (far > kb_lo + 1) far = kb_lo;"),
    ("return (c >= lo || c < sk) && c <= hi;", "return c >= lo || c < sk;"),
    ("return (j < far ? j : kb_lo + j - far) * kBlockN;", "return (j < far ? j : kb_lo + j) * kBlockN;"),
])
def test_the_check_rejects_planted_mistakes(tmp_path, old, new):
    src = open(os.path.join(CSRC, "swa_kernels.h")).read()
    assert src.count(old) == 1
    (tmp_path / "hdr").mkdir()
    (tmp_path / "hdr" / "swa_kernels.h").write_text(src.replace(old, new))
    r = check(tmp_path, tmp_path / "hdr")
    assert r.returncode == 1 and r.stdout.startswith("mismatch"), r.stdout
