"""Build libep.so (the C-ABI library of include/ep.h) in-tree with hipcc for gfx950, and
_tensor_ptr.so (the binding's tensor check, host code against torch's headers) with g++.

Every HIP source is compiled with packed-fp32 instructions disabled
(``-Xclang -target-feature -Xclang -packed-fp32-ops``); hipcc's host pass warns that
it does not know the feature, which is harmless.
"""
from __future__ import annotations

import concurrent.futures
import os
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libep.so")
TENSOR_PTR = os.path.join(PKG, "_tensor_ptr.so")
SOURCES = ["ep_abi.cpp", "layout.hip", "dispatch.hip", "restripe.hip", "combine.hip",
           "hbm_copy.hip", "rmsnorm.hip", "expert_rows.hip", "expert_ffn.hip",
           "expert_ffn_grad.hip"]
ARCH = "gfx950"
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CXX = os.environ.get("CXX", "g++")

CFLAGS = ["-x", "hip", f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-Wall",
          "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
          "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def _compile(src: str, verbose: bool, build_dir: str, defines) -> str:
    obj = os.path.join(build_dir, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *CFLAGS, *[f"-D{d}" for d in defines], "-c", os.path.join(CSRC, src),
           "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    noise = "is not a recognized feature for this target"
    msgs = "\n".join(l for l in (r.stdout + r.stderr).splitlines() if noise not in l)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{msgs}")
    if msgs.strip() and verbose:
        print(msgs, flush=True)
    return obj


def build_tensor_ptr(verbose: bool = False) -> str:
    import torch
    from torch.utils import cpp_extension

    cmd = [CXX, "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[a for p in cpp_extension.include_paths() for a in ("-isystem", p)],
           "-isystem", sysconfig.get_paths()["include"], os.path.join(CSRC, "tensor_ptr.cpp"),
           *[a for p in cpp_extension.library_paths() for a in (f"-L{p}", f"-Wl,-rpath,{p}")],
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-o", TENSOR_PTR + ".tmp"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{CXX} failed on tensor_ptr.cpp:\n{r.stdout}{r.stderr}")
    os.replace(TENSOR_PTR + ".tmp", TENSOR_PTR)
    return TENSOR_PTR


def build(verbose: bool = False, defines=(), lib: str = LIB, build_dir: str = BUILD) -> str:
    """Compile every source and link the library; always rebuilds. The package's own libep.so
    (the default) comes with _tensor_ptr.so, which the binding's calls need beside it; a
    library elsewhere is built alone. `defines` override the kernels' compile-time tile
    constants (NAME=VALUE strings)."""
    os.makedirs(build_dir, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, len(SOURCES))) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose, build_dir, defines), SOURCES))
    tmp = lib + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, lib)
    if lib == LIB:
        build_tensor_ptr(verbose)
    return lib


if __name__ == "__main__":
    print(build(verbose=True))
