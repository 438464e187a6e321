"""Build libprn.so (HIP, gfx950) in-tree with hipcc.

Usage: python -m nonlinear_rnn_amd.build   (or __graft_entry__.build())
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys
import tempfile
import time

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libprn.so")
SOURCES = ["prn_lib.hip", "proj.hip", "embed.hip", "block_norm.hip", "vocab_loss.hip"]
ARCH = os.environ.get("PRN_OFFLOAD_ARCH", "gfx950")

# Packed fp32 VALU instructions are disabled: plain fp32 code only.
HIP_FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-command-line-argument",
]


def hipcc() -> str:
    for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("hipcc not found (ROCm is required to build libprn)")


def build(verbose: bool = True) -> str:
    """Compile every source (side by side) and link them into libprn.so."""
    t0 = time.time()
    with tempfile.TemporaryDirectory(prefix="prn_build_") as tmp:
        objs = [os.path.join(tmp, s + ".o") for s in SOURCES]
        cmds = [[hipcc(), *HIP_FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", os.path.join(CSRC, s), "-o", o]
                for s, o in zip(SOURCES, objs)]
        if verbose:
            for c in cmds:
                print("[prn build]", " ".join(c), flush=True)
        with concurrent.futures.ThreadPoolExecutor(max_workers=min(len(cmds), os.cpu_count() or 1)) as pool:
            runs = list(pool.map(lambda c: subprocess.run(c, capture_output=True, text=True), cmds))
        out = LIB + ".tmp"
        if all(r.returncode == 0 for r in runs):
            runs.append(subprocess.run([hipcc(), *HIP_FLAGS, "-shared", "-o", out, *objs], capture_output=True,
                                       text=True))
    for r in runs:
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError(f"hipcc failed with exit code {r.returncode}")
        if verbose and r.stderr.strip():
            sys.stderr.write(r.stderr[-4000:])
    os.replace(out, LIB)
    if verbose:
        print(f"[prn build] {LIB} built in {time.time() - t0:.1f} s", flush=True)
    return LIB


if __name__ == "__main__":
    build()
