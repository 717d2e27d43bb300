"""Build libdspark.so (gfx950) in-tree with hipcc.

Usage: python -m draft_sampling_verification_w1_amd.build
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJDIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libdspark.so")
SOURCES = ["bias_pass.hip", "select.hip", "verify_aux.hip", "schedule.hip", "misc.hip", "acceptance.hip",
           "sts.hip", "check.hip", "logprobs.hip", "cache.hip",
           "cache_store.hip", "attend.hip", "attend4.hip", "api.hip"]

HIPCC_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    "-fvisibility=hidden",
    # no packed-fp32 instructions anywhere in device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I" + os.path.join(ROOT, "include"),
]


# Per-source flags.  These passes never produce or test a NaN (entries outside the
# vocabulary are -inf, a block whose maximum is -inf is left before any
# difference of infinities is formed, and keys and values of whole elements are
# finite by their contract); without NaNs to honour, the compiler drops the
# NaN-quieting v_max it otherwise puts in front of every maximum of matrix-core
# results.  attend4.hip is not among them: its blocks without a value are NaN.
EXTRA_FLAGS = {"bias_pass.hip": ["-fno-honor-nans"], "attend.hip": ["-fno-honor-nans"]}


def _hipcc() -> str:
    for c in (os.environ.get("HIPCC"), shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("hipcc not found")


def _compile(src: str) -> str:
    obj = os.path.join(OBJDIR, os.path.splitext(src)[0] + ".o")
    cmd = [_hipcc(), *HIPCC_FLAGS, *EXTRA_FLAGS.get(src, []), "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stderr}")
    return obj


def build() -> str:
    """Compile every HIP source and link libdspark.so; returns its path."""
    os.makedirs(OBJDIR, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [_hipcc(), "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build())
    sys.exit(0)
