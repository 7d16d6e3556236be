"""Builds libbsp.so (the C-ABI CUDA library) in-tree for sm_100a, and the
CPython binding of its fused GEMMs (_fused_binding.so, plain C++ over it).

    python -m block_scaled_precision_05_b200.csrc.build [--force] [--verbose]

The library needs nvcc and its host compiler alone; without torch, Python's
headers or g++ (run as a script: python block_scaled_precision_05_b200/csrc/build.py)
it is built without the binding.

Each .cu is compiled with nvcc (-gencode arch=compute_100a,code=sm_100a) in
parallel into _build/, then linked against the shared CUDA runtime (so the
library shares the process's runtime, device and streams with PyTorch).
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
PKG = os.path.dirname(HERE)
ROOT = os.path.dirname(PKG)
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(PKG, "libbsp.so")
BINDING = os.path.join(PKG, "_fused_binding.so")
BINDING_STAMP = os.path.join(BUILD_DIR, "fused_binding.stamp")  # what BINDING was compiled against
SOURCES = ["common.cu", "quantize.cu", "gemm.cu", "fused_gemm_nvfp4.cu", "fused_gemm_mxfp8.cu"]
HEADERS = ["activation.cuh", "bsp_device.cuh", "bsp_internal.h", "fused_gemm.cuh", "norm_stats.cuh", "per_device.h",
           "tensor_maps.h"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def cuda_lib_dir() -> str:
    return os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "lib64")


FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC",
    "--expt-relaxed-constexpr",
    "-Xptxas", "-warn-spills",
]


def _stale(out: str, deps: list[str]) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


# Per-source flags.  The quantizers must round every fp32 product and sum on its
# own (their results are compared bit for bit with an oracle that does), so no
# multiply-add contraction there: explicit fma calls stay fused, nothing else is.
SOURCE_FLAGS = {"quantize.cu": ["-fmad=false"]}


def _compile(src: str, verbose: bool, extra: list[str]) -> str:
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    deps = [os.path.join(HERE, src)] + [os.path.join(HERE, h) for h in HEADERS] + [os.path.join(INCLUDE, "bsp.h"),
                                                                                   os.path.abspath(__file__)]
    if _stale(obj, deps) or extra:
        cmd = [nvcc(), *FLAGS, *SOURCE_FLAGS.get(src, []), *extra, "-I", INCLUDE, "-I", HERE, "-c",
               os.path.join(HERE, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, flush=True)
    return obj


def binding_target() -> str:
    """The torch and Python that the binding is compiled against; the module holds it as `built_for`, and another torch or
    Python gets a binding of its own."""
    import torch

    return f"torch {torch.__version__} cxx11abi={int(torch._C._GLIBCXX_USE_CXX11_ABI)} {sys.implementation.cache_tag}"


def _binding_stale(deps: list[str]) -> bool:
    if _stale(BINDING, deps) or not os.path.exists(BINDING_STAMP):
        return True
    with open(BINDING_STAMP) as f:
        return f.read() != binding_target()


def binding_lacks() -> str | None:
    """What the binding's build needs and this machine has not; the library does without it."""
    if importlib.util.find_spec("torch") is None:
        return "torch"
    if shutil.which("g++") is None:
        return "g++"
    header = os.path.join(sysconfig.get_paths()["include"], "Python.h")
    return None if os.path.exists(header) else header


def _build_binding(verbose: bool) -> None:
    """csrc/fused_binding.cpp against torch's headers and libbsp.so (found next to it at run time)."""
    lacks = binding_lacks()
    if lacks is not None:
        print(f"libbsp.so is built; _fused_binding.so (the Python binding of the fused GEMMs) is not: no {lacks}",
              file=sys.stderr, flush=True)
        return
    import torch

    src = os.path.join(HERE, "fused_binding.cpp")
    if not _binding_stale([src, os.path.join(INCLUDE, "bsp.h"), os.path.abspath(__file__)]):
        return
    top = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(cuda_lib_dir()), "include")
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DBSP_BUILT_FOR="{binding_target()}"', "-I", INCLUDE, "-I", sysconfig.get_paths()["include"], "-I", os.path.join(top, "include"),
           "-I", os.path.join(top, "include", "torch", "csrc", "api", "include"), "-I", cuda, src, "-o", tmp,
           "-L", PKG, "-l:libbsp.so", "-L", os.path.join(top, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
           "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{os.path.join(top, 'lib')}"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for fused_binding.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    with open(BINDING_STAMP, "w") as f:
        f.write(binding_target())


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    """Compile every source for sm_100a and link libbsp.so; returns its path."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    extra = list(extra or [])
    if force:
        for f in os.listdir(BUILD_DIR):
            if f.endswith(".o"):
                os.remove(os.path.join(BUILD_DIR, f))
    with cf.ThreadPoolExecutor(len(SOURCES)) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose, extra), SOURCES))
    if force or extra or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc(), "-shared", "-cudart", "shared", "-o", tmp, *objs,
               "-Xlinker", f"-rpath,{cuda_lib_dir()}"]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    if force and os.path.exists(BINDING):
        os.remove(BINDING)
    _build_binding(verbose)
    return LIB


def main(argv=None) -> int:
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-v", action="store_true", help="print register/spill/smem usage")
    a = ap.parse_args(argv)
    extra = ["-Xptxas", "-v"] if a.ptxas_v else []
    print(build(force=a.force, verbose=a.verbose or a.ptxas_v, extra=extra))
    return 0


if __name__ == "__main__":
    sys.exit(main())
