"""The build of the binding's module (csrc/swa_torch.cpp), which the library does without: on the CPU."""
import os
import sys
import types

import pytest
import torch

import sliding_window_flash_gb300 as swa
from sliding_window_flash_gb300 import cache
from sliding_window_flash_gb300 import build


@pytest.fixture
def module(tmp_path, monkeypatch):
    """The module's place in a folder of its own; the library is there, or built once."""
    build.build()
    path = tmp_path / "_swa_torch.so"
    monkeypatch.setattr(build, "TORCH_PATH", str(path))
    return path


def compiler(monkeypatch, code):
    """`code`, Python, in the compiler's place, with `out` the file to make."""
    monkeypatch.setattr(build, "_torch_command", lambda nvcc, out: [sys.executable, "-c",
                                                                    f"import sys\nout = {out!r}\n{code}"])


def test_the_library_is_built_without_the_module(module, monkeypatch, capsys):
    compiler(monkeypatch, "open(out, 'w').write('half')\nsys.exit('no Python.h')")
    module.write_text("made for another torch")
    os.utime(module, (1, 1))
    assert os.path.exists(build.build())
    assert "no Python.h" in capsys.readouterr().err
    assert not module.exists() and not os.path.exists(str(module) + ".tmp")
    monkeypatch.setattr(build, "_torch_command", lambda nvcc, out: [str(module) + "-no-compiler", out])
    assert os.path.exists(build.build())
    assert "no-compiler" in capsys.readouterr().err and not module.exists()
    compiler(monkeypatch, "open(out, 'w').write('whole')")
    build.build()
    assert module.read_text() == "whole"


def test_a_library_that_does_not_compile_is_an_error(module, monkeypatch, tmp_path):
    bad = tmp_path / "bad.cu"
    bad.write_text("#error no kernel\n")
    compiler(monkeypatch, "open(out, 'w').write('whole')")
    monkeypatch.setattr(build, "sources", lambda: [str(bad)])
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path / "objects"))
    monkeypatch.setattr(build, "LIB_PATH", str(tmp_path / "libswa.so"))
    with pytest.raises(RuntimeError, match="no kernel"):
        build.build()
    assert not (tmp_path / "libswa.so").exists()


def test_the_module_is_made_again_for_another_torch(module, monkeypatch, tmp_path):
    """Also where the new torch's files are older than the module, as an installer may leave them."""
    for text in ("first", "second"):
        compiler(monkeypatch, f"open(out, 'w').write({text!r})")
        for _ in range(2):
            build.build()
            assert module.read_text() == text
    version = tmp_path / "version.py"
    version.write_text("")
    os.utime(version, (2**31, 2**31))
    monkeypatch.setattr(build, "_torch_version_file", lambda: str(version))
    module.write_text("old")
    build.build()
    assert module.read_text() == "second"


def test_the_command_names_torch_and_python(monkeypatch, tmp_path):
    command = build._torch_command(build._nvcc(), "x")
    assert f'-DSWA_BUILT_FOR="{build.built_for(torch.__version__)}"' in command
    (tmp_path / "version.py").write_text("__version__ = '9.8.7+cu1'\n")
    monkeypatch.setattr(build, "_torch_version_file", lambda: str(tmp_path / "version.py"))
    assert any("torch 9.8.7+cu1, " in arg for arg in build._torch_command(build._nvcc(), "x"))
    monkeypatch.setattr(build, "_torch_version_file", lambda: None)
    assert build._torch_command(build._nvcc(), "x") is None


def test_a_module_for_another_torch_is_not_used(monkeypatch):
    build.build()
    used = []
    fake = types.SimpleNamespace(use=lambda *at: used.append(at), pool=1, cache_attn=2, fwd=3, bwd=4)
    monkeypatch.setattr(swa, "_swa_torch", fake, raising=False)
    for other in (None, "torch 1.0, cpython-311", build.built_for(torch.__version__) + "d"):
        if other:
            fake.built_for = other
        way = cache._short_way()
        assert not used and all(way[n](1, 2, 3) is None for n in ("pool", "attn", "fwd", "bwd"))
    fake.built_for = build.built_for(torch.__version__)
    assert cache._short_way() == {"pool": 1, "attn": 2, "fwd": 3, "bwd": 4} and len(used) == 1


def test_the_short_way_asks_nobody_else(monkeypatch, tmp_path):
    """Torch's names need no library, and the library that is used is the one in its place, whatever stands for
    it elsewhere."""
    def other(*_):
        raise RuntimeError("another library")

    build.build()
    monkeypatch.setattr(cache, "_entry", other)
    monkeypatch.setattr(swa, "load", other)
    names = cache._Torch()
    assert names.f32 is torch.float32 and names.empty is torch.empty and "fwd" not in names.__dict__
    assert names.fwd is swa._swa_torch.fwd
    monkeypatch.setattr(swa, "library_path", lambda: str(tmp_path / "libswa.so"))
    assert cache._Torch().fwd(1, 2, 3) is None


def test_the_module_that_is_built_is_used():
    build.build()
    fwd = cache._t.fwd
    assert swa._swa_torch.built_for == build.built_for(torch.__version__)
    assert fwd is swa._swa_torch.fwd
