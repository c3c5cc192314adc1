"""Builds the gfx950 shared library libtopk_transform.so in-tree with hipcc."""
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
LIB_NAME = "libtopk_transform.so"
LIB_PATH = os.path.join(PKG, LIB_NAME)

SOURCES = ["topk_kernels.hip", "topk_api.cpp", "indexer_kernels.hip", "indexer_api.cpp", "cache_kernels.hip",
           "attend_kernels.hip", "prefill_kernels.hip", "latent_api.cpp"]

HIPCC_FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    # packed fp32 VALU forms stay off: plain float code only
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall",
    "-Wno-unused-command-line-argument",
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", "hipcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "hipcc"


def _run(cmd) -> str:
    res = subprocess.run(cmd, capture_output=True, text=True)
    noise = "is not a recognized feature for this target"
    err = "\n".join(l for l in res.stderr.splitlines() if noise not in l)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed ({res.returncode}):\n{err}")
    return err


def build(verbose: bool = False) -> str:
    """Compiles every source (side by side) and links them into LIB_PATH;
    returns the path.  Always recompiles."""
    tmp = LIB_PATH + ".tmp"
    with tempfile.TemporaryDirectory() as objs:
        jobs = [[hipcc(), *HIPCC_FLAGS, "-c", "-I", INCLUDE, "-I", CSRC, os.path.join(CSRC, s), "-o",
                 os.path.join(objs, s + ".o")] for s in SOURCES]
        link = [hipcc(), *HIPCC_FLAGS, "-shared", *(j[-1] for j in jobs), "-o", tmp]
        with ThreadPoolExecutor(min(len(jobs), 8)) as pool:
            errs = list(pool.map(_run, jobs))
        errs.append(_run(link))
    if verbose:
        for cmd in (*jobs, link):
            print(" ".join(cmd), flush=True)
        text = "\n".join(e for e in errs if e.strip())
        if text:
            print(text, file=sys.stderr)
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose=True))
