"""Build the gfx950 HIP library libmxfp8.so in-tree with hipcc."""

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_PATH = os.path.join(HERE, "libmxfp8.so")
SOURCES = ["mx_api.cpp", "mx_quant.hip", "mx_pc.hip", "mx_gemm.hip", "mx_small.hip", "mx_probe.hip", "mx_noalloc.hip",
           "mx_fp4_quant.hip", "mx_fp4_small.hip", "mx_fp4_gemm.hip", "mx_fp4_mid.hip",
           "mx_norm.hip", "mx_block_norm.hip", "mx_experts.hip", "mx_experts_tile.hip", "mx_experts_few.hip", "mx_route.hip"]

# Device code is built without packed-FP32 instructions (v_pk_*_f32).
HIP_FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-shared",
    "-Xclang",
    "-target-feature",
    "-Xclang",
    "-packed-fp32-ops",
    "-parallel-jobs=8",  # sources at a time
]


def build(verbose=False):
    """Compile every source for gfx950 into LIB_PATH (always recompiles)."""
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    tmp = LIB_PATH + ".tmp"
    cmd = [hipcc, *HIP_FLAGS, "-I", INCLUDE, "-I", CSRC, "-o", tmp] + [os.path.join(CSRC, s) for s in SOURCES]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"hipcc failed with exit code {res.returncode}")
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose=True))
