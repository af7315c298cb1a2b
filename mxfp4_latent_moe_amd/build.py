"""Build the gfx950 HIP library in-tree: mxfp4_latent_moe_amd/lib/libmoe_latent.so.

    python -m mxfp4_latent_moe_amd.build

Every source is compiled for gfx950 only, with packed fp32 ops disabled
(`-Xclang -target-feature -Xclang -packed-fp32-ops`).  The assembly of the
kernels that pace their LDS reads by hand is checked (asm_check.py): a build in
which a register is used before its read has landed fails.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

from .asm_check import unsafe_reads

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIBDIR = os.path.join(PKG, "lib")
LIB = os.path.join(LIBDIR, "libmoe_latent.so")
BUILD = os.path.join(ROOT, "_build")

SOURCES = ["abi.hip", "gemm.hip", "stream.hip", "grouped_stream.hip", "prefill.hip", "route.hip",
           "permute.hip", "combine.hip", "mx8.hip", "dense.hip", "reap.hip", "prefill_pl.hip",
           "block.hip", "fp8.hip", "few.hip"]
CHECKED = ["dense.hip", "fp8.hip", "prefill.hip", "prefill_pl.hip"]  # issue LDS reads in inline assembly
HIPCC_FLAGS = [
    "-O3", "-std=c++17", "--offload-arch=gfx950", "-fPIC",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found; the HIP library cannot be built")


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    out = "\n".join(line for line in r.stdout.splitlines() if "packed-fp32-ops" not in line)
    if r.returncode != 0:
        raise RuntimeError(f"command failed ({r.returncode}): {' '.join(cmd)}\n{out}")
    if verbose and out.strip():
        print(out)


def _check(src):
    path = os.path.join(BUILD, os.path.splitext(src)[0] + "-hip-amdgcn-amd-amdhsa-gfx950.s")
    with open(path) as f:
        bad = unsafe_reads(f.read())
    if bad:
        raise RuntimeError(f"{src}: registers used before their LDS read has landed:\n"
                           + "\n".join(f"  {name}, line {no}: {text}" for name, no, text in bad[:20]))


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    cc = hipcc()
    objs = []
    cmds = []
    for src in SOURCES:
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        objs.append(obj)
        keep = ["-save-temps=obj"] if src in CHECKED else []
        cmds.append([cc, *HIPCC_FLAGS, *keep, "-I", INCLUDE, "-I", CSRC, "-c", os.path.join(CSRC, src), "-o", obj])
    with ThreadPoolExecutor(min(len(cmds), os.cpu_count() or 1)) as ex:
        list(ex.map(lambda c: _run(c, verbose), cmds))
    for src in CHECKED:
        _check(src)
    tmp = LIB + ".tmp"
    _run([cc, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp], verbose)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
