"""Compile the CUDA sources of this package into libmbw.so (sm_103a only), and
the binding's hot calls into _fast.so (g++, against the headers of PyTorch).

One nvcc process per translation unit, run in parallel, then one link step.
The library is built in-tree (memory_bound_weight_gb300/libmbw.so) and loaded
with ctypes by the binding.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmbw.so")
GEN_LIB = os.path.join(PKG, "libmbw_inputs.so")
FAST = os.path.join(PKG, "_fast.so")
FAST_FOR = os.path.join(BUILD, "_fast.for")  # the Python and PyTorch that it was built for

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
                     "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]

# translation units of libmbw.so (the product) and of the input generator
LIB_SOURCES = ["abi.cu", "plan.cu", "gemv_simt.cu", "gemv_mma.cu", "gemv_tma.cu", "gemv_lat.cu", "gemm_tc.cu",
               "gemv_awq_batch.cu", "quantize.cu", "kv4_cache.cu", "kv4_attention.cu",
               "kv4_attention_tc.cu", "logprobs.cu", "quantize_fp8.cu", "gemm_fp8.cu", "gemv_fp8.cu"]
GEN_SOURCES = ["gen_inputs.cu"]


def _nvcc() -> str:
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def _stale(out: str, deps: list[str]) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def _headers() -> list[str]:
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    return hs + [os.path.join(INCLUDE, "mbw.h")]


def _compile(src: str, ptxas_v: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    if _stale(obj, [src] + _headers()):
        cmd = [_nvcc(), *NVCC_FLAGS, "-c", src, "-o", obj]
        if ptxas_v:
            cmd += ["-Xptxas", "-v"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if ptxas_v:
            sys.stderr.write(r.stderr)
    return obj


def _link(objs: list[str], out: str) -> None:
    if not _stale(out, objs):
        return
    tmp = out + ".tmp"
    cmd = [_nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)


def _here() -> str:
    """This Python and this installation of PyTorch, which need not be imported for it."""
    import importlib.util

    spec = importlib.util.find_spec("torch")
    at = spec.origin if spec and spec.origin else None
    return f"{sys.implementation.cache_tag} {at} {os.stat(at).st_mtime_ns if at else 0}"


def _built_for() -> str:
    try:
        with open(FAST_FOR) as f:
            return f.read()
    except OSError:
        return ""


def _fast() -> None:
    """_fast.so; where it cannot be compiled (no PyTorch or no headers of it or of Python, no g++) the binding marshals every
    call in Python."""
    src = os.path.join(CSRC, "fast_calls.cpp")
    if not _stale(FAST, [src, os.path.join(INCLUDE, "mbw.h")]) and _built_for() == _here():
        return
    try:
        import sysconfig

        import torch

        at, inc = os.path.dirname(torch.__file__), sysconfig.get_path("include")
        cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
               f'-DMBW_BUILT_FOR="{sys.implementation.cache_tag} torch {torch.__version__}"',
               "-I", os.path.join(at, "include"), "-I", inc, "-I", os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include"),
               "-I", INCLUDE, src, "-o", FAST + ".tmp", "-L", os.path.join(at, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10",
               "-lc10_cuda"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        why = r.stderr[-2000:] if r.returncode != 0 else None
    except (ImportError, OSError) as e:
        why = str(e)
    if why is not None:
        sys.stderr.write(f"_fast.so is not built, calls are marshalled in Python:\n{why}\n")
        if os.path.exists(FAST):
            os.remove(FAST)
        return
    os.replace(FAST + ".tmp", FAST)
    with open(FAST_FOR, "w") as f:
        f.write(_here())


def build(ptxas_v: bool = False) -> str:
    """Build libmbw.so, libmbw_inputs.so and _fast.so; returns the path of libmbw.so."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = [os.path.join(CSRC, f) for f in LIB_SOURCES + GEN_SOURCES]
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        fast = ex.submit(_fast)
        objs = list(ex.map(lambda s: _compile(s, ptxas_v), srcs))
        fast.result()
    _link(objs[: len(LIB_SOURCES)], LIB)
    _link(objs[len(LIB_SOURCES):], GEN_LIB)
    return LIB


if __name__ == "__main__":
    print(build(ptxas_v="-v" in sys.argv))
