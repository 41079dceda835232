"""Builds libdg.so (the gfx950 kernels and their C ABI) in the package
directory with hipcc. Run as `python -m moe_grouped_gemm_amd.build`."""

from __future__ import annotations

import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libdg.so")

SOURCES = ["dg_kernel.hip", "dg_kernel_deep.hip", "dg_kernel_kgrouped.hip", "dg_kernel_fp4.hip", "dg_kernel_mx.hip",
           "dg_quantize_fp4.hip", "dg_ceiling.hip",
           "dg_moe_route.hip", "dg_moe_glu.hip", "dg_moe_norm.hip",
           "dg_moe_experts.hip", "dg_api.cpp", "dg_moe_api.cpp"]

HIPCC_FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-shared",
    # Packed FP32 instructions stay off: the compiler would otherwise pair
    # the promotion FMAs into v_pk_fma_f32.
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # MFMA results in VGPRs, so the promotion FMAs read them directly.
    "-mllvm", "-amdgpu-mfma-vgpr-form",
    "-Wno-unused-command-line-argument",
]


def hipcc() -> str:
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    path = os.path.join(rocm, "bin", "hipcc")
    return path if os.path.exists(path) else "hipcc"


def build(verbose: bool = False) -> str:
    """Compile every source into libdg.so (always recompiles)."""
    tmp = LIB + ".tmp"
    cmd = [hipcc(), *HIPCC_FLAGS, "-I", os.path.join(ROOT, "include"),
           *[os.path.join(CSRC, s) for s in SOURCES], "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed ({res.returncode}):\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
