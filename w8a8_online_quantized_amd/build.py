"""Builds libcider.so (the HIP kernels and the C ABI of include/cider.h) for
gfx950 with hipcc, in-tree next to this file.

Usage: python -m w8a8_online_quantized_amd.build [-v]
"""
from __future__ import annotations

import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libcider.so")
SOURCES = ["cider_api.hip", "cider_quant.hip", "cider_gemm.hip", "cider_mv.hip", "cider_probe.hip",
           "cider_grouped.hip", "cider_moe_plan.hip", "cider_norm.hip", "cider_rope.hip", "cider_kv4_cache.hip",
           "cider_kv4_attention.hip"]

HIPCC_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared",
    # packed fp32 VALU instructions stay off for every kernel of this library
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    return "hipcc"


def build(verbose: bool = False) -> str:
    """Compile every HIP source into libcider.so; returns the library path."""
    srcs = [os.path.join(CSRC, s) for s in SOURCES]
    tmp = LIB + ".tmp"
    cmd = [hipcc(), *HIPCC_FLAGS, "-I", os.path.join(ROOT, "include"), *srcs, "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    noise = "is not a recognized feature for this target"
    msgs = "\n".join(l for l in (res.stdout + res.stderr).splitlines() if noise not in l)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed ({res.returncode}):\n{msgs}")
    if verbose and msgs.strip():
        print(msgs)
    # every symbol of the library's own namespace must be defined in it (a
    # kernel whose host-side launch stub was not emitted links fine and only
    # fails when the library is loaded)
    nm = subprocess.run(["nm", "-D", "--undefined-only", tmp], capture_output=True, text=True)
    if nm.returncode == 0:
        missing = [l.split()[-1] for l in nm.stdout.splitlines() if "cider" in l]
        if missing:
            os.remove(tmp)
            raise RuntimeError("libcider.so has undefined symbols of its own: " + ", ".join(missing))
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
