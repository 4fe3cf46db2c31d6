"""Builds libzero.so (the C-ABI library and its HIP kernels) for gfx950, in-tree.

Usage: python -m zero_sharded_mixed_bucketed_amd._build
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libzero.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

# -ffp-contract=off and correctly rounded fp32 division and square root: every
# operation of the Adam update rounds once, as the update is specified.  Packed
# fp32 instructions are left out of code generation altogether.
HIP_FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-Wall",
    "-ffp-contract=off", "-fhip-fp32-correctly-rounded-divide-sqrt",
    "-fno-gpu-flush-denormals-to-zero",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def sources():
    return sorted(glob.glob(os.path.join(HERE, "csrc", "*.hip")))


def _run(cmd, what: str) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(f"hipcc failed building {what}")


def build(verbose: bool = False) -> str:
    """Compiles every source to an object, side by side, and links them."""
    tmp = LIB + f".tmp{os.getpid()}"
    inc = ["-I", os.path.join(ROOT, "include"), "-I", os.path.join(HERE, "csrc")]
    with tempfile.TemporaryDirectory() as d:
        objs = [os.path.join(d, os.path.basename(s) + ".o") for s in sources()]
        cmds = [[HIPCC, *HIP_FLAGS, *inc, "-c", s, "-o", o] for s, o in zip(sources(), objs)]
        if verbose:
            print("\n".join(" ".join(c) for c in cmds), flush=True)
        jobs = max(1, min(8, len(cmds), len(os.sched_getaffinity(0))))
        with concurrent.futures.ThreadPoolExecutor(jobs) as pool:
            for f in [pool.submit(_run, c, c[-3]) for c in cmds]:
                f.result()
        _run([HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp],
             "libzero.so")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
