"""Builds libcider.so (the HIP kernels and the C ABI of include/cider.h) for
gfx950 with hipcc, in-tree next to this file.

Usage: python -m w8a8_online_quantized_amd.build [-v]
"""
from __future__ import annotations

import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libcider.so")
SOURCES = ["cider_api.hip", "cider_quant.hip", "cider_gemm.hip", "cider_mv.hip", "cider_probe.hip",
           "cider_grouped.hip", "cider_moe_plan.hip", "cider_norm.hip", "cider_rope.hip", "cider_kv4_cache.hip",
           "cider_kv4_attention.hip"]

HIPCC_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
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
    """Compile every HIP source into libcider.so; returns the library path.

    The sources are compiled side by side (each is independent device code),
    those with the most kernels first.
    """
    tmp = LIB + ".tmp"

    def run(args) -> None:
        cmd = [hipcc(), *HIPCC_FLAGS, *args]
        if verbose:
            print(" ".join(cmd), flush=True)
        res = subprocess.run(cmd, capture_output=True, text=True)
        noise = "is not a recognized feature for this target"
        msgs = "\n".join(l for l in (res.stdout + res.stderr).splitlines() if noise not in l)
        if res.returncode != 0:
            raise RuntimeError(f"hipcc failed ({res.returncode}):\n{msgs}")
        if verbose and msgs.strip():
            print(msgs)

    with tempfile.TemporaryDirectory() as objs:
        def compile_one(source: str) -> str:
            obj = os.path.join(objs, source + ".o")
            run(["-c", "-I", os.path.join(ROOT, "include"), os.path.join(CSRC, source), "-o", obj])
            return obj

        jobs = int(os.environ.get("MAX_JOBS", "") or min(8, os.cpu_count() or 1))
        with ThreadPoolExecutor(max(1, min(jobs, 8))) as pool:
            todo = [pool.submit(compile_one, s) for s in reversed(SOURCES)]
            linked = [t.result() for t in todo]
        run(["-shared", *reversed(linked), "-o", tmp])
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
