"""Build libbsk.so in-tree from csrc/ with nvcc for sm_103a.

The translation units compile in parallel (one nvcc per file), then link into
``bf16_gemm_skinny_gb300/_build/libbsk.so``.  ``_calls.so`` beside it is the Python
module that calls some of its entry points.  Rebuilds only when a source or header
is newer than either.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(BUILD_DIR, "libbsk.so")
CALLS_PATH = os.path.join(BUILD_DIR, "_calls.so")
CALLS_SOURCE = os.path.join(CSRC, "py_calls.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", f"-I{INCLUDE}", "-Xptxas", "-v"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + [CALLS_SOURCE] + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def is_stale() -> bool:
    if not os.path.exists(LIB_PATH) or not os.path.exists(CALLS_PATH):
        return True
    t = min(os.path.getmtime(LIB_PATH), os.path.getmtime(CALLS_PATH))
    return any(os.path.getmtime(d) > t for d in _deps())


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link libbsk.so and _calls.so; returns the library's path."""
    if not force and not is_stale():
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(src):
        name = os.path.splitext(os.path.basename(src))[0]
        obj = os.path.join(BUILD_DIR, name + ".o")
        python = [f"-I{sysconfig.get_paths()['include']}"] if src == CALLS_SOURCE else []
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *python, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        log = os.path.join(BUILD_DIR, name + ".ptxas.log")
        with open(log, "w") as f:
            f.write(r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr[-4000:]}")
        return obj

    with cf.ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        *objs, calls = ex.map(compile_one, _sources() + [CALLS_SOURCE])

    def link(path, args):
        tmp = path + f".tmp{os.getpid()}"
        r = subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *args], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("link failed:\n" + r.stderr[-4000:])
        os.replace(tmp, path)

    link(LIB_PATH, [*objs, "-lcudart"])
    link(CALLS_PATH, [calls, "-cudart", "none", f"-L{BUILD_DIR}", "-lbsk", "-Xlinker", "-rpath,$ORIGIN"])
    if verbose:
        print(f"built {LIB_PATH}")
    return LIB_PATH


if __name__ == "__main__":
    build(force=True, verbose=True)
