"""Build libsp24.so (the C-ABI library with its HIP kernels) for gfx950, in-tree.

Each source compiles to an object under <repo>/_build with hipcc (in parallel), then one hipcc link
produces structured_sparse_gemm_sp24_amd/libsp24.so. hipcc cross-compiles, so no GPU is needed. The native
marshalling of the 8-bit operators (binding/fp8_binding.cpp) and of the layer operators (binding/layer_binding.cpp) compiles
with g++ against torch's headers into the extension modules _fp8_binding.so and _layer_binding.so, which link to libsp24.so
beside them.
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libsp24.so")
BUILD_DIR = os.path.join(ROOT, "_build")
BINDINGS = ("fp8_binding", "layer_binding")  # binding/<name>.cpp -> _<name>.so

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"
COMMON = ["-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}", "-Wall", "-Wno-unused-function",
          "-I", os.path.join(ROOT, "include")]
# device code: no packed-fp32 instructions; no fast-math anywhere (the epilogues rely on IEEE rounding)
DEVICE_ONLY = ["-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-ffp-contract=on"]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.hip"))) + sorted(glob.glob(os.path.join(CSRC, "*.cpp")))


def _compile(src: str) -> str:
    obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
    cmd = [HIPCC] + COMMON + (DEVICE_ONLY if src.endswith(".hip") else []) + ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stderr}")
    return obj


def _compile_binding(name: str) -> str:
    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    src = os.path.join(PKG, "binding", name + ".cpp")
    obj = os.path.join(BUILD_DIR, name + ".cpp.o")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-fvisibility=hidden", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "include"),
           "-isystem", sysconfig.get_paths()["include"], "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {src}:\n{r.stderr}")
    return obj


def _link_binding(name: str, obj: str) -> str:
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    so = os.path.join(PKG, f"_{name}.so")
    tmp = so + ".tmp"
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L" + PKG, "-lsp24", "-L" + lib, "-ltorch_python", "-ltorch", "-ltorch_cpu",
           "-ltorch_hip", "-lc10", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of the binding failed:\n{r.stderr}")
    os.replace(tmp, so)
    return so


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    srcs = sources()
    workers = max(1, min(len(srcs), int(os.environ.get("MAX_JOBS", "8"))))
    with concurrent.futures.ThreadPoolExecutor(workers) as ex:
        bindings = [ex.submit(_compile_binding, name) for name in BINDINGS]
        objs = list(ex.map(_compile, srcs))
        binding_objs = [b.result() for b in bindings]
    tmp = LIB + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-Wl,-soname,libsp24.so", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    built = [LIB] + [_link_binding(name, obj) for name, obj in zip(BINDINGS, binding_objs)]
    if verbose:
        print("built " + ", ".join(built))
    return LIB


if __name__ == "__main__":
    build(verbose=True)
