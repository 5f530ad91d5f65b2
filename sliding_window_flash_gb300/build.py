"""Build libswa.so in-tree: every csrc/*.cu compiled for sm_103a in parallel, then linked; and beside it
_swa_torch.so, the binding's short way to it (csrc/swa_torch.cpp, with torch's headers).

    python -m sliding_window_flash_gb300.build [--verbose] [--ptxas-info]

Objects go to sliding_window_flash_gb300/_build/, the library to sliding_window_flash_gb300/libswa.so.
nvcc and the CUDA toolkit are needed, for the second a C++ compiler and torch (no GPU): the build runs
the same on x86_64 and aarch64.  The library does without the second: where it does not compile, the compiler's
output goes to stderr, an older one is removed, and the binding takes the Python way.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG_DIR, "_build")
LIB_PATH = os.path.join(PKG_DIR, "libswa.so")
TORCH_SRC = os.path.join(CSRC, "swa_torch.cpp")
TORCH_PATH = os.path.join(PKG_DIR, "_swa_torch.so")

ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]
COMMON_FLAGS = ARCH_FLAGS + [
    "-O3",
    "-std=c++17",
    "-lineinfo",
    "--expt-relaxed-constexpr",
    "-Xcompiler",
    "-fPIC,-O2",
    "-I" + INCLUDE,
    "-I" + CSRC,
]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libswa.so")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def built_for(torch_version: str) -> str:
    """What the binding's module is compiled for: it reads torch's and Python's objects by their layouts."""
    return f"torch {torch_version}, {sysconfig.get_config_var('SOABI')}"


def _torch_version_file():
    """torch/version.py of the torch that would be imported, or None."""
    spec = importlib.util.find_spec("torch")
    path = spec and os.path.join(spec.submodule_search_locations[0], "version.py")
    return path if path and os.path.exists(path) else None


def _torch_command(nvcc: str, out: str):
    """The compiler's command for the binding's module: torch is found, not imported.  None without torch."""
    path = _torch_version_file()
    if path is None:
        return None
    with open(path) as f:
        version = re.search(r"^__version__ = ['\"](.*)['\"]", f.read(), re.M)
    torch = os.path.dirname(path)
    lib = os.path.join(torch, "lib")
    include = [INCLUDE, os.path.join(torch, "include"),
               os.path.join(torch, "include", "torch", "csrc", "api", "include"),
               os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include"),
               sysconfig.get_paths()["include"]]
    return [os.environ.get("CXX") or shutil.which("g++") or "c++", "-O2", "-std=c++17", "-fPIC", "-shared",
            "-fvisibility=hidden", f'-DSWA_BUILT_FOR="{built_for(version.group(1) if version else "?")}"', *["-I" + d for d in include], TORCH_SRC, "-o", out, "-L" + lib,
            "-Wl,-rpath," + lib, "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]


def _module_stale(command) -> bool:
    """Whether the binding's module has to be compiled: its sources, or the torch that it was compiled for,
    are newer, or the command that made it, which names torch's and Python's versions and paths, was another."""
    deps = [TORCH_SRC, _torch_version_file()] + glob.glob(os.path.join(INCLUDE, "*.h"))
    if _stale(TORCH_PATH, filter(None, deps)) or not os.path.exists(TORCH_PATH + ".stamp"):
        return True
    with open(TORCH_PATH + ".stamp") as f:
        return f.read() != "\n".join(command)


def _put_module(made: str, r) -> None:
    """The binding's module in its place; where the compiler failed, none, and why on stderr."""
    if r.returncode == 0:
        os.replace(made, TORCH_PATH)
        with open(TORCH_PATH + ".stamp", "w") as f:
            f.write("\n".join(r.args))
        return
    for path in (made, TORCH_PATH, TORCH_PATH + ".stamp"):
        if os.path.exists(path):
            os.remove(path)
    sys.stderr.write(f"no {os.path.basename(TORCH_PATH)} (calls take some microseconds more on the host): the "
                     f"compiler failed for {TORCH_SRC}:\n{r.stdout}\n{r.stderr}\n")


def build(verbose: bool = False, ptxas_info: bool = False, force: bool = False) -> str:
    """Compile (if needed) and return the path of libswa.so."""
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    headers = _headers()
    srcs = sources()
    objs = []
    jobs = []
    for src in srcs:
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or ptxas_info or _stale(obj, [src] + headers):
            cmd = [nvcc] + COMMON_FLAGS + (["-Xptxas", "-v"] if ptxas_info else []) + ["-c", src, "-o", obj]
            jobs.append((src, cmd))
    short, short_job = TORCH_PATH + ".tmp", None
    command = _torch_command(nvcc, short)
    if command and (force or _module_stale(command)):
        short_job = TORCH_SRC, command

    def run(job):
        src, cmd = job
        if verbose:
            print(" ".join(cmd), flush=True)
        try:
            r = subprocess.run(cmd, capture_output=True, text=True)
        except OSError as e:  # no such compiler
            r = subprocess.CompletedProcess(cmd, 127, "", str(e))
        return src, r

    every = ([short_job] if short_job else []) + jobs
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(every), os.cpu_count() or 4))) as ex:
        done = list(ex.map(run, every))
    for src, r in done:
        if src == TORCH_SRC:
            _put_module(short, r)
        elif r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose or ptxas_info:
            sys.stdout.write(r.stdout + r.stderr)
    if force or jobs or _stale(LIB_PATH, objs):
        tmp = LIB_PATH + ".tmp"
        cmd = [nvcc] + ARCH_FLAGS + ["-shared", "-o", tmp] + objs
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true")
    ap.add_argument("--force", action="store_true")
    args = ap.parse_args()
    print(build(verbose=args.verbose, ptxas_info=args.ptxas_info, force=args.force))
