"""Compile libsn.so (the HIP kernels and the C ABI) for gfx950, in-tree.

Usage: python -m schnet_cfconv_force_amd.build
"""
from __future__ import annotations

import concurrent.futures
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
OUT = os.path.join(HERE, "libsn.so")
BUILD_DIR = os.path.join(ROOT, "_build")

SOURCES = ["neighbors.hip", "graph.hip", "mlp.hip", "filter.hip", "attention_fwd.hip", "attention_bwd.hip", "norm.hip", "context.hip",
           "rotary.hip", "cache.hip", "cache_attend.hip", "state.hip", "api.hip"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"
FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-fPIC", "-std=c++17",
    # never emit packed fp32 instructions (v_pk_fma_f32 and friends)
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
]
# accumulators of 16 registers stay whole where paths join: taken apart, they
# are copied back into consecutive registers every tile
WHOLE_VECTORS = ["-mllvm", "-amdgpu-codegenprepare-break-large-phis=false"]
# the neighbour predicate must round every operation on its own
PER_FILE = {"neighbors.hip": ["-ffp-contract=off"],
            "attention_fwd.hip": WHOLE_VECTORS, "attention_bwd.hip": WHOLE_VECTORS}


def _compile(src: str) -> str:
    obj = os.path.join(BUILD_DIR, src.replace(".hip", ".o"))
    cmd = [HIPCC, *FLAGS, *PER_FILE.get(src, []), "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stderr}")
    return obj


def build(verbose: bool = True) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, len(SOURCES))) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = OUT + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, OUT)
    if verbose:
        print(f"built {OUT}")
    return OUT


if __name__ == "__main__":
    build()
    sys.exit(0)
