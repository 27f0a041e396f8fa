"""Build libkda.so (HIP kernels + C ABI) for gfx950 with hipcc, in-tree."""
from __future__ import annotations

import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libkda.so")
SOURCES = ["api.hip", "debug.hip", "gate.hip", "decode.hip", "decode_gated.hip", "prefill.hip", "prep.hip",
           "state.hip", "shortconv.hip", "backward.hip", "linattn_api.hip", "linattn_walk.hip",
           "linattn_decode.hip", "layernorm.hip", "gatedrec_api.hip", "gatedrec_scan.hip",
           "gatedrec_backward.hip", "gatedrec_decode.hip", "rmsnorm.hip"]
ARCH = os.environ.get("KDA_OFFLOAD_ARCH", "gfx950")


def hipcc() -> str:
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    return os.path.join(rocm, "bin", "hipcc")


def _run(cmd, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("hipcc failed building libkda.so")


def build_library(verbose: bool = False) -> str:
    """Compile every HIP source, several at a time, into one shared library; returns its path."""
    tmp = LIB + ".tmp%d" % os.getpid()
    cc = [hipcc(), "--offload-arch=" + ARCH, "-fPIC"]
    flags = [
        "-O3", "-std=c++17",
        # packed fp32 VALU ops stay off: hipcc otherwise forms them from plain float code
        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
        "-munsafe-fp-atomics", "-Wno-unused-command-line-argument",
        "-I", os.path.join(ROOT, "include"), "-I", CSRC,
    ]
    jobs = int(os.environ.get("MAX_JOBS") or min(8, os.cpu_count() or 1))
    with tempfile.TemporaryDirectory(prefix="build_", dir=HERE) as to:
        objects = [os.path.join(to, s + ".o") for s in SOURCES]
        with ThreadPoolExecutor(max(1, jobs)) as pool:
            list(pool.map(lambda so: _run(cc + flags + ["-c", os.path.join(CSRC, so[0]), "-o", so[1]],
                                          verbose), zip(SOURCES, objects)))
        _run(cc + ["-shared", "-o", tmp] + objects, verbose)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build_library(verbose=True))
