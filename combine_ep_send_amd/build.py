"""Build libepdc.so (HIP, gfx950) in-tree with hipcc.

    python -m combine_ep_send_amd.build

Flags: -O3 for gfx950 only; ``-ffp-contract=off`` so the combine's fp32
product and sum are rounded separately; packed-fp32 instructions disabled.
fp32 division stays correctly rounded and denormals are kept (the HIP
defaults), which the fp8 scale and quotient rely on.
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libepdc.so")
SOURCES = ["scan.hip", "fused.hip", "rows.hip", "api.hip", "expert.hip", "grad.hip",
           "expert_api.hip", "norm.hip", "route.hip", "gate.hip",
           "router_api.hip"]
ARCH = "gfx950"

HIPCC_FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-shared",
    "-ffp-contract=off",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall",
    "-Wno-unused-command-line-argument",
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (ROCm is required to build libepdc.so)")


def build(verbose: bool = False) -> str:
    """Compile every HIP source, side by side, into combine_ep_send_amd/libepdc.so."""
    tmp = LIB + ".tmp"

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        proc = subprocess.run(cmd, capture_output=True, text=True)
        if proc.returncode != 0:
            sys.stderr.write(proc.stdout + proc.stderr)
            raise RuntimeError(f"hipcc failed with status {proc.returncode}")

    with tempfile.TemporaryDirectory() as objects:
        objs = [os.path.join(objects, s + ".o") for s in SOURCES]
        flags = [f for f in HIPCC_FLAGS if f != "-shared"] + ["-I", os.path.join(ROOT, "include")]
        cc = hipcc()
        with ThreadPoolExecutor(min(8, os.cpu_count() or 1)) as pool:
            list(pool.map(lambda so: run([cc, *flags, "-c", "-o", so[1],
                                          os.path.join(CSRC, so[0])]), zip(SOURCES, objs)))
        run([cc, *HIPCC_FLAGS, "-o", tmp, *objs])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
