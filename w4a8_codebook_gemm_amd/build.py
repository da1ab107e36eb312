"""Compile the HIP sources for gfx950 into three shared libraries: csrc/ into libw4a8.so (the
quantised layer, exporting the C ABI declared in include/w4a8.h), csrc/attn/ into
libw4a8_attn.so (the attention operators, include/w4a8_attn.h) and csrc/serve/ into
libw4a8_serve.so (the serving operators, include/w4a8_serve.h).

Each source is compiled to an object in _build/ (in parallel), then linked.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build", "w4a8")
LIB = os.path.join(PKG, "libw4a8.so")
ATTN_CSRC = os.path.join(CSRC, "attn")
ATTN_LIB = os.path.join(PKG, "libw4a8_attn.so")
SERVE_CSRC = os.path.join(CSRC, "serve")
SERVE_LIB = os.path.join(PKG, "libw4a8_serve.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-fvisibility=hidden",
    # every fp32 operation stays one IEEE operation unless written as fmaf(): the int8
    # activations and the quantiser's outputs are compared bit-exact
    "-ffp-contract=off",
    # no packed fp32 arithmetic
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
    f"-I{os.path.join(ROOT, 'include')}",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.hip")))


def attn_sources():
    return sorted(glob.glob(os.path.join(ATTN_CSRC, "*.hip")))


def serve_sources():
    return sorted(glob.glob(os.path.join(SERVE_CSRC, "*.hip")))


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [HIPCC, *FLAGS, "-c", src, "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    if verbose and r.stderr.strip():
        print(r.stderr, flush=True)
    return obj


def _link(objs, lib: str, verbose: bool) -> None:
    tmp = lib + ".tmp%d" % os.getpid()
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, lib)


def build(verbose: bool = False, jobs: int = 8) -> str:
    os.makedirs(BUILD, exist_ok=True)
    parts = [(sources(), LIB), (attn_sources(), ATTN_LIB), (serve_sources(), SERVE_LIB)]
    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        futs = [[ex.submit(_compile, s, verbose) for s in srcs] for srcs, _ in parts]
        objs = [[f.result() for f in fs] for fs in futs]
    for (_, lib), o in zip(parts, objs):
        _link(o, lib, verbose)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
