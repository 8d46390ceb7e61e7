"""Build the HIP library libdeltarule.so for gfx950 (in-tree, next to this file).

    python -m delta_rule_linear_amd.build

Each .hip translation unit is compiled to an object in parallel, then linked
into one shared library exporting the C ABI of include/deltarule.h.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libdeltarule.so")
SOURCES = ["dr_abi.hip", "dr_chunk.hip", "dr_scan16.hip", "dr_prep16.hip", "dr_prepcg16.hip", "dr_decode.hip",
           "dr_bwd.hip", "dr_bwd16.hip", "dr_linattn_abi.hip", "dr_linattn.hip", "dr_linattn32.hip", "dr_layernorm.hip",
           "dr_seqops_abi.hip", "dr_rmsnorm.hip", "dr_rmsnorm_bwd.hip", "dr_conv.hip", "dr_scan.hip", "dr_scan_bwd.hip"]
ARCH = os.environ.get("DR_OFFLOAD_ARCH", "gfx950")

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
    "-I", os.path.join(ROOT, "include"),
    # no packed-fp32 VALU instructions in device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def _compile(src: str, outdir: str) -> str:
    obj = os.path.join(outdir, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stderr}")
    return obj


def build(verbose: bool = False) -> str:
    outdir = os.path.join(HERE, "_build")
    os.makedirs(outdir, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(lambda s: _compile(s, outdir), SOURCES))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
