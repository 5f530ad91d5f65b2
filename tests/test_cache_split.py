"""CPU check of how the cache attention divides its work (swa_cache_split.h) against brute force.

tests/cache_split_check.cpp includes the library's own header.  Mutation checks: copies of the header
with a planted mistake must be rejected."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sliding_window_flash_gb300", "csrc")


def _run(tmp_path, header_dir):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("needs a host C++ compiler")
    exe = str(tmp_path / "cache_split_check")
    subprocess.run([cxx, "-std=c++17", "-O2", f"-I{header_dir}",
                    os.path.join(ROOT, "tests", "cache_split_check.cpp"), "-o", exe],
                   check=True, capture_output=True, text=True)
    return subprocess.run([exe], capture_output=True, text=True, timeout=120)


def test_split_matches_brute_force(tmp_path):
    r = _run(tmp_path, CSRC)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout + r.stderr


@pytest.mark.parametrize("old,new", [
    ("at >= window ? at - window + 1 : 0", "at >= window ? at - window : 0"),
    ("(len + n - 1) / ck", "(len + n) / ck"),
    ("(i < extra ? i : extra)", "(i <= extra ? i : extra - 1)"),
    ("const int64_t longer = (size + 1) * extra;", "const int64_t longer = size * extra;"),
    ("((x | d) >> 32) == 0", "true"),
    ("if (first[mid] * per <= x)", "if (first[mid] * per < x)"),
    ("used = n > 1 ? quotient(total + n - 1, n) : total;", "used = total + n;"),
    ("used < 1 ? 1 :", "false ? 1 :"),
    ("2 * part + (begins ? 1 : 0)", "part + (begins ? 1 : 0)"),
])
def test_split_check_rejects_planted_mistakes(tmp_path, old, new):
    src = open(os.path.join(CSRC, "swa_cache_split.h")).read()
    assert src.count(old) == 1, old
    hdr = tmp_path / "hdr"
    hdr.mkdir()
    (hdr / "swa_cache_split.h").write_text(src.replace(old, new))
    r = _run(tmp_path, str(hdr))
    assert r.returncode == 1 and r.stdout.startswith("failed"), r.stdout
