"""Build libblr.so (the HIP kernels and the C ABI of include/blr.h) in-tree
with hipcc for gfx950. Run as `python -m binary_rank_linear_amd.build`."""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SOURCES = [os.path.join(HERE, "csrc", f) for f in ("blr_kernels.hip", "blr_route.hip", "blr_adapters.hip",
                                                     "blr_adapters_backward.hip", "blr_api.hip")]
HEADERS = [os.path.join(HERE, "csrc", f) for f in ("blr_internal.h", "blr_plan.h", "blr_vec.h", "blr_adapters.h")] + \
    [os.path.join(ROOT, "include", "blr.h")]
LIB = os.path.join(HERE, "libblr.so")
ARCH = "gfx950"


def hipcc() -> str:
    for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("hipcc not found (ROCm is required to build libblr.so)")


def flags() -> list[str]:
    return [
        f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-shared",
        # no packed-f32 VALU instructions (v_pk_*_f32) anywhere in device code
        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
        "-Wall", "-Wno-unused-command-line-argument",
        "-I", os.path.join(ROOT, "include"),
    ]


def build(verbose: bool = False) -> str:
    def run(cmd: list[str]):
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError(f"hipcc failed with status {r.returncode}")

    # the sources side by side, then one link
    with tempfile.TemporaryDirectory() as d, ThreadPoolExecutor(len(SOURCES)) as pool:
        objects = [os.path.join(d, os.path.basename(src) + ".o") for src in SOURCES]
        list(pool.map(lambda so: run([hipcc()] + [f for f in flags() if f != "-shared"] + ["-c", "-o", so[1], so[0]]),
                      zip(SOURCES, objects)))
        tmp = LIB + ".tmp"
        run([hipcc()] + flags() + ["-o", tmp] + objects)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
