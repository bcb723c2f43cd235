"""Build step of libddtree.so: hipcc for gfx950, in-tree."""

from __future__ import annotations

import glob
import os
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OBJ = os.path.join(HERE, "build")
LIB = os.path.join(HERE, "libddtree.so")

HIPCC_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    # No packed-FP32 instructions anywhere in the device code.
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # A wave's atomic add of per-lane amounts to one address: one DPP scan and
    # one atomic instead of a scalar loop over the active lanes.
    "-mllvm", "-amdgpu-atomic-optimizer-strategy=DPP",
]


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(HERE, "csrc", "*")) +
                  [os.path.join(ROOT, "include", "ddtree.h")])


def _run(cmd: list[str]) -> str:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed ({r.returncode}):\n{r.stderr}")
    return r.stderr


def build_library(verbose: bool = False) -> str:
    """Compile every csrc/*.hip (they include the kernel headers), side by side, and link
    them into libddtree.so."""
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    os.makedirs(OBJ, exist_ok=True)
    with tempfile.TemporaryDirectory(dir=OBJ) as tmp:
        jobs = []
        for src in sorted(glob.glob(os.path.join(CSRC, "*.hip"))):
            obj = os.path.join(tmp, os.path.basename(src) + ".o")
            jobs.append((obj, [hipcc, *HIPCC_FLAGS, "-c", "-I", os.path.join(ROOT, "include"), src,
                               "-o", obj]))
        with ThreadPoolExecutor(len(jobs)) as pool:
            said = list(pool.map(_run, [cmd for _, cmd in jobs]))
        lib = os.path.join(tmp, "libddtree.so")
        said.append(_run([hipcc, "--offload-arch=gfx950", "-shared", "-fPIC",
                          *[obj for obj, _ in jobs], "-o", lib]))
        os.replace(lib, LIB)
    if verbose and any(t.strip() for t in said):
        print("\n".join(said))
    return LIB
