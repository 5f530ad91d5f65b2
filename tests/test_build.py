"""The build of the binding's module (csrc/swa_torch.cpp), which the library does without: on the CPU."""
import os
import sys

import pytest

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
