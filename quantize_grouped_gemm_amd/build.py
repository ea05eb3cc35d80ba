"""Builds libmxfp8.so (the HIP kernels + C ABI) for gfx950 with hipcc, and
_lmhost.so (the C++ host path of lm, against torch's headers) with g++.

    python -m quantize_grouped_gemm_amd.build [--resource-usage]

Objects go to _build/ at the repository root; the libraries are written next
to this file so they are found in-tree.
"""

import argparse
import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libmxfp8.so")
HOST_LIB = os.path.join(PKG, "_lmhost.so")
SOURCES = ["mx_quant.hip", "mx_gemm.hip", "mx_pad_hp.hip", "mx_fp8.hip", "mx_norm.hip", "mx_swiglu_ck.hip",
           "mx_logprob.hip", "mx_abi.cpp", "mx_lm_abi.cpp"]
ARCH = "gfx950"

# -packed-fp32-ops keeps the compiler from emitting packed float32 VALU ops.
FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-fPIC", "-std=c++17", "-Wall",
    "-Wno-unused-function", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
]


def hipcc():
    exe = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(exe):
        raise RuntimeError("hipcc not found: the ROCm toolchain is required to build libmxfp8.so")
    return exe


def _compile(src, resource_usage=False):
    obj = os.path.join(BUILD, src + ".o")
    cmd = [hipcc(), *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    if resource_usage and src.endswith(".hip"):
        cmd.append("-Rpass-analysis=kernel-resource-usage")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{r.stderr}")
    return obj, r.stderr


def build(verbose=False, resource_usage=False):
    """Compile every source and link libmxfp8.so. Always recompiles."""
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(8, len(SOURCES))) as ex:
        results = list(ex.map(lambda s: _compile(s, resource_usage), SOURCES))
    objs = [o for o, _ in results]
    if verbose or resource_usage:
        for src, (_, err) in zip(SOURCES, results):
            if err.strip():
                print(f"--- {src}\n{err}", file=sys.stderr)
    tmp = LIB + ".tmp"
    cmd = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    build_host()
    return LIB


def build_host():
    """Compile _lmhost.so. It finds libmxfp8.so beside itself and torch's
    libraries in the process (torch is imported first)."""
    import torch
    root = os.path.dirname(torch.__file__)
    tmp = HOST_LIB + ".tmp"
    cmd = ["g++", "-O2", "-fPIC", "-shared", "-std=c++17", "-w", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", os.path.join(root, "include"), "-I", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-I", os.path.join(os.path.dirname(os.path.dirname(hipcc())), "include"),
           "-I", sysconfig.get_paths()["include"], os.path.join(CSRC, "lm_host.cpp"), "-o", tmp,
           "-L", PKG, "-l:libmxfp8.so", "-L", os.path.join(root, "lib"), "-lc10", "-lc10_hip", "-ltorch_cpu",
           "-ltorch_hip", "-ltorch_python", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on lm_host.cpp:\n{r.stderr}")
    os.replace(tmp, HOST_LIB)
    return HOST_LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--resource-usage", action="store_true")
    ap.add_argument("-v", "--verbose", action="store_true")
    args = ap.parse_args()
    print(build(args.verbose, args.resource_usage))
