"""Build the HIP library libkda.so in-tree with hipcc for gfx950."""
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
LIB = os.path.join(PKG, "libkda.so")
SOURCES = ["kda_abi.hip", "kda_prefill.hip", "kda_replay.hip",
           "kda_linear_abi.hip", "kda_linear_step.hip", "kda_linear_chunk.hip", "kda_cache.hip",
           "kda_block_abi.hip", "kda_scan.hip", "kda_block_norm.hip", "kda_act.hip"]

HIPCC_FLAGS = [
    "-O3", "-std=c++17", "-fPIC", "-shared", "--offload-arch=gfx950",
    # keep the compiler from emitting packed-fp32 VALU instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-fvisibility=hidden", "-Wall", "-Wno-unused-function",
]


def hipcc() -> str:
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    return os.path.join(rocm, "bin", "hipcc")


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    res = subprocess.run(cmd, capture_output=True, text=True)
    noise = "is not a recognized feature for this target"
    err = "\n".join(x for x in res.stderr.splitlines() if noise not in x)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed:\n{err}")
    if verbose and err.strip():
        print(err, file=sys.stderr)


def build(verbose: bool = False) -> str:
    """Compile every source (always, side by side) and link libkda.so."""
    tmp = LIB + ".tmp"
    flags = [x for x in HIPCC_FLAGS if x != "-shared"]
    jobs = min(len(SOURCES), int(os.environ.get("MAX_JOBS", 0)) or os.cpu_count() or 1, 8)
    with tempfile.TemporaryDirectory() as d, ThreadPoolExecutor(jobs) as pool:
        objects = [os.path.join(d, s + ".o") for s in SOURCES]
        # the longest first
        order = sorted(range(len(SOURCES)), key=lambda i: -os.path.getsize(os.path.join(CSRC, SOURCES[i])))
        done = [pool.submit(_run, [hipcc(), *flags, "-I", INCLUDE, "-I", CSRC, "-c", os.path.join(CSRC, SOURCES[i]), "-o", objects[i]],
                            verbose) for i in order]
        for f in done:
            f.result()
        _run([hipcc(), "-fPIC", "-shared", "--offload-arch=gfx950", *objects, "-o", tmp], verbose)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
