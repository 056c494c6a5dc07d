"""Build libmuon.so (HIP kernels + C ABI) in-tree for gfx950.

    python -m matrix_aware_optimizer_amd.build

The library is compiled with hipcc straight from ``csrc/*.hip`` into
``matrix_aware_optimizer_amd/libmuon.so``, one process per source.  Packed fp32
instructions are disabled for all device code (``-packed-fp32-ops``).
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
REPO_DIR = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(REPO_DIR, "include")
LIB_PATH = os.path.join(PKG_DIR, "libmuon.so")
SOURCES = ["elementwise.hip", "ns.hip", "dion.hip", "fp8.hip", "blocks.hip", "int8.hip", "gated.hip"]
ARCH = os.environ.get("MUON_OFFLOAD_ARCH", "gfx950")


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found: the HIP toolchain is required to build libmuon")


def compile_flags() -> list:
    return [
        f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-shared",
        "-mcode-object-version=5", f"-I{INCLUDE}", f"-I{CSRC}",
        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
        "-Wno-unused-result",
    ]


def _run(cmd: list, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    proc = subprocess.run(cmd, capture_output=True, text=True)
    # hipcc's host pass warns that it does not know the packed-fp32 feature; drop that line
    noise = "is not a recognized feature for this target"
    err = "\n".join(l for l in proc.stderr.splitlines() if noise not in l)
    if proc.returncode != 0:
        raise RuntimeError(f"hipcc failed ({proc.returncode}):\n{err}")
    if err.strip() and verbose:
        print(err, file=sys.stderr)


def build(verbose: bool = False) -> str:
    """Compile every HIP source and link libmuon.so; returns the library path."""
    flags = [f for f in compile_flags() if f != "-shared"]
    tmp = LIB_PATH + ".tmp"
    with tempfile.TemporaryDirectory() as objects:
        outs = [os.path.join(objects, s + ".o") for s in SOURCES]
        with ThreadPoolExecutor(min(len(SOURCES), os.cpu_count() or 1)) as pool:
            list(pool.map(lambda so: _run([hipcc()] + flags + ["-c", os.path.join(CSRC, so[0]), "-o", so[1]], verbose),
                          zip(SOURCES, outs)))
        _run([hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC"] + outs + ["-o", tmp], verbose)
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose=True))
