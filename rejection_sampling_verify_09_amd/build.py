"""Build libspecverify.so (the gfx950 HIP kernels and the C ABI) in-tree."""
from __future__ import annotations

import concurrent.futures
import os
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libspecverify.so")
SOURCES = ["sv_kernels.hip", "sv_api.hip", "sv_lmhead.hip", "sv_norm.hip", "sv_layer_norm.hip", "sv_linear.hip",
           "sv_adjust.hip", "sv_top.hip", "sv_distill.hip", "sv_dynk.cpp"]
ARCH = "gfx950"

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-ffp-contract=off",
    # no packed fp32 (v_pk_*_f32) instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-result",
]


def _run(cmd, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(f"hipcc failed with exit code {r.returncode}")


def _jobs() -> int:
    """Compilers at a time: MAX_JOBS if that is a number above 0, else the processors, at most 8 and a source each."""
    try:
        n = int(os.environ.get("MAX_JOBS", ""))
    except ValueError:
        n = 0
    return max(1, min(len(SOURCES), n if n > 0 else os.cpu_count() or 1, 8))


def build(verbose: bool = False) -> str:
    """Compile every source, side by side, and link them into libspecverify.so; returns its path."""
    tmp = LIB + ".tmp"
    with tempfile.TemporaryDirectory() as d:
        objs = [os.path.join(d, s + ".o") for s in SOURCES]
        with concurrent.futures.ThreadPoolExecutor(_jobs()) as pool:
            list(pool.map(lambda so: _run([HIPCC, *FLAGS, f"-I{INCLUDE}", f"-I{CSRC}", "-c", os.path.join(CSRC, so[0]), "-o",
                                           so[1]], verbose), zip(SOURCES, objs)))
        _run([HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs], verbose)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
