"""Builds the HIP library (libhisparse.so) in-tree with hipcc for gfx950."""
from __future__ import annotations

import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libhisparse.so")
SOURCES = [os.path.join(CSRC, f) for f in ("hs_api.cpp", "hs_kernels.hip", "hs_tokens.hip", "hs_attend.hip",
                                           "hs_prompt.hip", "hs_heads.hip", "hs_score.hip",
                                           "hs_select.hip")]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    # packed fp32 instructions are kept out of every kernel
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function", "-Wno-unused-command-line-argument",
    "-I", INCLUDE, "-I", CSRC,
]

# The attention and score kernels: matrix instructions whose results other instructions read (scores) write to the ordinary registers
MFMA_FLAGS = ["-mllvm", "-amdgpu-mfma-vgpr-form=1"]


def flags_of(src: str):
    return FLAGS + (MFMA_FLAGS if os.path.basename(src) in ("hs_attend.hip", "hs_prompt.hip", "hs_score.hip") else [])


def build(verbose: bool = False) -> str:
    def run(cmd):
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            sys.stderr.write(res.stdout + res.stderr)
            raise RuntimeError("hipcc failed to build libhisparse.so")
        if verbose:
            sys.stderr.write(res.stderr)

    # the sources side by side, then one link
    with tempfile.TemporaryDirectory() as objects:
        out = [os.path.join(objects, os.path.basename(src) + ".o") for src in SOURCES]
        with ThreadPoolExecutor(len(SOURCES)) as pool:
            list(pool.map(lambda so: run([HIPCC, *flags_of(so[0]), "-c", so[0], "-o", so[1]]), zip(SOURCES, out)))
        tmp = LIB + ".tmp"
        run([HIPCC, *FLAGS, "-shared", "-o", tmp, *out])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
