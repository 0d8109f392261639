"""Build libbakron.so (HIP for gfx950) in-tree with hipcc.

    python -m kronecker_factored_gptq_amd.build

Objects go to _build/ at the repository root; the shared library to
kronecker_factored_gptq_amd/_lib/libbakron.so.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIBDIR = os.path.join(PKG, "_lib")
LIB = os.path.join(LIBDIR, "libbakron.so")

SOURCES = ["abi.cpp", "abi_product.cpp", "abi_experts.cpp", "product_kernels.hip", "plane_kernels.hip",
           "fp8_kernels.hip", "expert_kernels.hip",
           "entropy_kernels.hip", "solve_kernels.hip", "band_kernels.hip", "factor_kernels.hip", "gemm64.hip", "loss_kernels.hip",
           "scale_kernels.hip", "gram_kernels.hip", "antidiag_kernels.hip"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"
COMMON = [
    f"--offload-arch={ARCH}", "-O3", "-fPIC", "-std=c++17",
    # never generate packed-fp32 (v_pk_*_f32) instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
    f"-I{INCLUDE}", f"-I{CSRC}",
]


# per-source options: MFMA accumulators in ordinary VGPRs (the leaf sweep
# reads its accumulator every in-tile step, and accumulation registers would
# need a copy per read; measured slightly faster for the band products too)
EXTRA = {"fp8_kernels.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"],
         "solve_kernels.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"],
         "band_kernels.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"],
         "antidiag_kernels.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"]}


def _compile(src: str, verbose: bool) -> str:
    path = os.path.join(CSRC, src)
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC] + COMMON + EXTRA.get(src, []) + ["-x", "hip", "-c", path, "-o", obj]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    r = subprocess.run(cmd, capture_output=True, text=True)
    msgs = "\n".join(l for l in (r.stdout + r.stderr).splitlines()
                     if "packed-fp32-ops" not in l and "not a recognized feature" not in l)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{msgs}")
    if verbose and msgs.strip():
        print(msgs, file=sys.stderr)
    return obj


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(8, len(SOURCES))) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stdout + r.stderr)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
