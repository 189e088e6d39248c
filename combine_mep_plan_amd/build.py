"""Ahead-of-time build of libmep.so for gfx950 with hipcc.

    python -m combine_mep_plan_amd.build

Flags: -O3, wave64 gfx950 code only, no fast-math and no FMA contraction
(the kernels spell out every fused multiply-add they want), packed-fp32 ops
disabled in the device pass.
"""

from __future__ import annotations

import concurrent.futures
import glob
import os
import subprocess
import sys
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libmep.so")

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-ffp-contract=off",
    "-fno-fast-math",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall",
    "-Wno-unused-command-line-argument",
]


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.hip"))) + \
        sorted(glob.glob(os.path.join(CSRC, "*.cpp")))


def _hipcc(args: list[str], verbose: bool) -> None:
    cmd = [HIPCC, *FLAGS, *args]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    # the host pass does not know the device-only target feature; drop that note
    noise = "'-packed-fp32-ops' is not a recognized feature"
    err = "\n".join(l for l in r.stderr.splitlines() if noise not in l)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed ({r.returncode}):\n{err}")
    if err.strip() and verbose:
        print(err, file=sys.stderr)


def build(verbose: bool = False) -> str:
    """Compiles every source, several at a time, and links them."""
    tmp = LIB + ".tmp"
    with tempfile.TemporaryDirectory() as objects:
        jobs = [(src, os.path.join(objects, os.path.basename(src) + ".o")) for src in sources()]
        workers = min(8, len(os.sched_getaffinity(0)), len(jobs))
        with concurrent.futures.ThreadPoolExecutor(workers) as pool:
            list(pool.map(lambda j: _hipcc(["-I", os.path.join(ROOT, "include"), "-I", CSRC, "-c",
                                            j[0], "-o", j[1]], verbose), jobs))
        _hipcc(["-shared", *(o for _, o in jobs), "-o", tmp], verbose)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
