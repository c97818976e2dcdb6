"""Build libbsk.so in-tree from csrc/ with nvcc for sm_103a.

The translation units compile in parallel (one nvcc per file), then link into
``bf16_gemm_skinny_gb300/_build/libbsk.so``.  ``_calls`` beside it is the Python
module that calls some of its entry points, compiled for (and named after) the
interpreter that builds it; the library itself needs no Python, and is built also where
the interpreter's headers are missing.  Each is rebuilt only when one of its sources or
headers is newer.
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
CALLS_PATH = os.path.join(BUILD_DIR, "_calls" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
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


def _headers():
    return glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def _python_include() -> str | None:
    """The folder of this interpreter's Python.h, or None where its headers are not installed."""
    path = sysconfig.get_paths()["include"]
    return path if os.path.exists(os.path.join(path, "Python.h")) else None


def _older(target, deps) -> bool:
    return not os.path.exists(target) or any(os.path.getmtime(d) > os.path.getmtime(target) for d in deps)


def _lib_stale() -> bool:
    return _older(LIB_PATH, _sources() + _headers())


def _calls_stale() -> bool:
    """False where the module cannot be built: the library needs no Python."""
    return _python_include() is not None and _older(CALLS_PATH, [CALLS_SOURCE] + _headers())


def is_stale() -> bool:
    return _lib_stale() or _calls_stale()


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link libbsk.so, then the module _calls; returns the library's path."""
    sources = _sources() if force or _lib_stale() else []
    module = _python_include() is not None and (force or _calls_stale())
    if not sources and not module:
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(src):
        name = os.path.splitext(os.path.basename(src))[0]
        obj = os.path.join(BUILD_DIR, name + ".o")
        python = [f"-I{_python_include()}"] if src == CALLS_SOURCE else []
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *python, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        log = os.path.join(BUILD_DIR, name + ".ptxas.log")
        with open(log, "w") as f:
            f.write(r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr[-4000:]}")
        return obj

    def link(path, args):
        tmp = path + f".tmp{os.getpid()}"
        r = subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *args], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("link failed:\n" + r.stderr[-4000:])
        os.replace(tmp, path)

    with cf.ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        calls = ex.submit(compile_one, CALLS_SOURCE) if module else None
        objs = list(ex.map(compile_one, sources))
        if objs:
            link(LIB_PATH, [*objs, "-lcudart"])
        if module:
            link(CALLS_PATH, [calls.result(), "-cudart", "none", f"-L{BUILD_DIR}", "-lbsk", "-Xlinker", "-rpath,$ORIGIN"])
    if verbose:
        print(f"built {LIB_PATH}")
    return LIB_PATH


if __name__ == "__main__":
    build(force=True, verbose=True)
