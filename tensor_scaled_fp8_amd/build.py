"""Build libfp8lin.so (all HIP sources, gfx950 only) and the compiled binding
of the block-scaled and serving operators (_block_binding.so, host code against torch)
in-tree.

    python -m tensor_scaled_fp8_amd.build [--jobs N]

Each .hip file is compiled to an object with hipcc in parallel, then linked
into tensor_scaled_fp8_amd/lib/libfp8lin.so. Packed FP32 instructions are
disabled for the device code (-target-feature -packed-fp32-ops)."""
from __future__ import annotations

import argparse
import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "lib")
BUILD_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(OUT_DIR, "libfp8lin.so")
BINDING = os.path.join(PKG, "_block_binding.so")
SOURCES = ["api.hip", "amax.hip", "cast.hip", "gemm.hip", "adam.hip", "block_quant.hip", "block_swiglu.hip",
           "block_gemm.hip", "block_serve.hip", "block_api.hip", "cache_store.hip", "cache_attention.hip", "fp4_quant.hip",
           "fp4_serve.hip", "serve_api.hip"]
BINDING_SOURCES = ["block_binding.cpp", "serve_binding.cpp"]
ARCH = "gfx950"

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CXX = os.environ.get("CXX", "g++")
CFLAGS = ["-O3", "-std=c++17", f"--offload-arch={ARCH}", "-fPIC", f"-I{INCLUDE}",
          "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
          "-Wall", "-Wno-unused-function"]


def _compile(src: str) -> str:
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *CFLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stderr}")
    return obj


def _compile_binding(src: str) -> str:
    """A source of the binding to an object, with the C++ ABI that torch was built with."""
    import torch
    from torch.utils.cpp_extension import include_paths
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    inc = [*include_paths(), "/opt/rocm/include", INCLUDE, sysconfig.get_paths()["include"]]
    cmd = [CXX, "-O2", "-std=c++17", "-fPIC", "-Wall", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *[f"-I{p}" for p in inc],
           "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{CXX} failed for {src}:\n{r.stderr}")
    return obj


def _link_binding(objs: list) -> None:
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + ".tmp"
    # not linked with the library: it takes the entry points of the one that is loaded
    cmd = [CXX, "-shared", *objs, "-o", tmp, f"-L{lib}", "-ltorch", "-ltorch_cpu", "-ltorch_python", "-lc10", "-lc10_hip",
           "-ldl", f"-Wl,-rpath,{lib}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of the binding failed:\n{r.stderr}")
    os.replace(tmp, BINDING)


def build(jobs: int = 4, verbose: bool = False) -> str:
    os.makedirs(OUT_DIR, exist_ok=True)
    os.makedirs(BUILD_DIR, exist_ok=True)
    with ThreadPoolExecutor(max_workers=max(1, jobs)) as ex:
        nodes = [ex.submit(_compile_binding, s) for s in BINDING_SOURCES]
        objs = list(ex.map(_compile, SOURCES))
        nodes = [n.result() for n in nodes]
    tmp = LIB + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    _link_binding(nodes)
    if verbose:
        print(f"built {LIB} and {BINDING}")
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--jobs", type=int, default=4)
    a = ap.parse_args()
    build(a.jobs, verbose=True)
    sys.exit(0)
