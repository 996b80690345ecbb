"""Build ``libdg.so`` (the C-ABI library) in-tree with nvcc for sm_103a.

One translation unit per kernel family, compiled in parallel, then linked
into ``fp16_tensor_core_gb300/_build/libdg.so`` against the shared CUDA
runtime (the same one PyTorch loads).  ``dg_python``, a small C module that
reads the arguments of the serving calls and of those around a layer's
products, is compiled with gcc and Python's headers.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(OUT_DIR, "libdg.so")
# Argument marshalling for Python; the name carries the interpreter's ABI, so
# that another interpreter builds and loads its own.
NATIVE = os.path.join(OUT_DIR, "dg_python" + sysconfig.get_config_var("EXT_SUFFIX"))

SOURCES = ["dg_api.cu", "k_scale.cu", "k_gemv.cu", "k_gemv_mma.cu", "k_gemm_tc.cu", "k_gemm_tc2.cu",
           "k_gemm_skinny.cu", "dg_static.cu", "k_kvcache.cu", "k_attn_decode.cu",
           "k_attn_prefix.cu", "k_norm.cu", "k_activate.cu",
           "k_gemm_tc_fused.cu", "k_gemm_tc2_fused.cu", "k_gemm_skinny_fused.cu", "k_epilogue.cu"]
HEADERS = ["dg_ptx.cuh", "dg_internal.h", "gemm_common.cuh", "attn_common.cuh", "prefix_barriers.h",
           "activation.cuh", "row_common.cuh", "gemm_tc_kernel.cuh", "gemm_pair_kernel.cuh",
           "gemm_skinny_kernel.cuh", "gemm_smem.h"]

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
              "--expt-relaxed-constexpr", "-Xptxas", "-warn-spills"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _deps():
    yield os.path.join(INCLUDE, "dg.h")
    yield __file__
    for h in HEADERS:
        yield os.path.join(CSRC, h)


def _stale(obj: str, src: str) -> bool:
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    return any(os.path.getmtime(p) > t for p in (src, *_deps()))


def _compile(src: str, verbose_ptxas: bool) -> str:
    obj = os.path.join(OUT_DIR, os.path.splitext(src)[0] + ".o")
    path = os.path.join(CSRC, src)
    if _stale(obj, path) or verbose_ptxas:
        cmd = [nvcc(), *ARCH, *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", path, "-o", obj]
        if verbose_ptxas:
            cmd[1:1] = ["-Xptxas", "-v"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose_ptxas:
            print(r.stdout, r.stderr)
    return obj


def _native_missing() -> str:
    """What the marshalling module needs and this machine lacks ("" if nothing)."""
    include = sysconfig.get_paths()["include"]
    if not os.path.exists(os.path.join(include, "Python.h")):
        return f"Python.h (looked in {include})"
    return "" if shutil.which("gcc") else "gcc"


def _build_native(force: bool) -> None:
    """dg_python, for the serving calls (rotary positions, cache, attention) and
    those around a layer's products (norm, activation, fused products) from
    Python.  libdg and everything else need only nvcc: without a C compiler or
    Python's headers this is left out with a warning, and these calls raise
    when they are made."""
    missing = _native_missing()
    if missing:
        warnings.warn(f"{missing} not found: the serving calls (dg_rope, dg_kv_append, dg_kv_read, dg_attn_decode) and "
                      "those around a layer's products (dg_rmsnorm, dg_rmsnorm_e4m3, dg_rmsnorm_e4m3_amax, "
                      "dg_rmsnorm_grad, dg_activate, dg_activate_grad, dg_fp8_gemm_fused, dg_hgemm_fused) cannot be "
                      "made from Python")
        return
    src = os.path.join(CSRC, "dg_python.c")
    deps = (src, os.path.join(INCLUDE, "dg.h"), __file__)
    if not force and os.path.exists(NATIVE) and all(
            os.path.getmtime(p) <= os.path.getmtime(NATIVE) for p in deps):
        return
    tmp = NATIVE + f".tmp{os.getpid()}"
    cmd = ["gcc", "-O2", "-shared", "-fPIC", "-I", INCLUDE, "-I", sysconfig.get_paths()["include"], src,
           "-o", tmp, "-lm"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"gcc failed for dg_python.c:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, NATIVE)


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Compile the CUDA sources and link libdg.so; return the library path."""
    os.makedirs(OUT_DIR, exist_ok=True)
    if force:
        for s in SOURCES:
            o = os.path.join(OUT_DIR, os.path.splitext(s)[0] + ".o")
            if os.path.exists(o):
                os.remove(o)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose_ptxas), SOURCES))
    if force or not os.path.exists(LIB) or any(
            os.path.getmtime(o) > os.path.getmtime(LIB) for o in objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc(), *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs,
               "-Xlinker", "-rpath=/usr/local/cuda/lib64"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    _build_native(force)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
