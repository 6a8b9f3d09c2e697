"""Build libternary_gemm.so in-tree with hipcc for gfx950."""
from __future__ import annotations

import os
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SRC = os.path.join(PKG, "csrc", "ternary_gemm.hip")
SRCS = [SRC, os.path.join(PKG, "csrc", "prep.hip"), os.path.join(PKG, "csrc", "block.hip"),
        os.path.join(PKG, "csrc", "int8.hip")]
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libternary_gemm.so")
# measurement probes for bench.py (a store floor and MFMA-only loops), not
# part of the GEMM library
PROBE_SRC = os.path.join(PKG, "csrc", "roofline.hip")
PROBE_LIB = os.path.join(PKG, "libtgemm_roofline.so")
ARCH = "gfx950"


def hipcc_cmd(out: str, *args) -> list[str]:
    return [
        "hipcc", f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
        # no packed-fp32 instructions in device code
        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
        "-I", INCLUDE, *args, "-o", out,
    ]


def _run(cmd, verbose):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("hipcc failed:\n" + r.stdout + r.stderr)
    if verbose:
        print(r.stderr)


def build(verbose: bool = False) -> str:
    """Compile the HIP library and the probe library (always; the sources side
    by side) and atomically replace the old ones."""
    with tempfile.TemporaryDirectory() as objs, ThreadPoolExecutor(4) as pool:
        obj = {src: os.path.join(objs, os.path.basename(src) + ".o") for src in (*SRCS, PROBE_SRC)}
        for done in [pool.submit(_run, hipcc_cmd(obj[src], "-c", src), verbose) for src in obj]:
            done.result()
        for lib, srcs in ((LIB, SRCS), (PROBE_LIB, [PROBE_SRC])):
            tmp = lib + ".tmp"
            _run(hipcc_cmd(tmp, "-shared", *(obj[src] for src in srcs)), verbose)
            os.replace(tmp, lib)
    return LIB


if __name__ == "__main__":
    print(build())
