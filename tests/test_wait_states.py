"""Wait states that the compiler cannot place inside inline asm, checked in the built library's device code."""
import os
import re
import shutil
import subprocess

import pytest

from matrix_aware_optimizer_amd import build as _build


def objdump():
    for cand in (shutil.which("llvm-objdump"), "/opt/rocm/llvm/bin/llvm-objdump"):
        if cand and os.path.exists(cand):
            return cand
    pytest.skip("llvm-objdump not found")


def device_code(tmp_path):
    """The instructions of every kernel of libmuon.so, one list for each source."""
    tool, lib = objdump(), str(tmp_path / "libmuon.so")
    if not os.path.exists(_build.LIB_PATH):
        _build.build()
    shutil.copy(_build.LIB_PATH, lib)
    subprocess.run([tool, "--offloading", lib], check=True, capture_output=True, cwd=tmp_path)
    parts = sorted(p for p in os.listdir(tmp_path) if "amdgcn" in p)
    assert len(parts) == len(_build.SOURCES)
    for part in parts:
        text = subprocess.run([tool, "-d", "--no-show-raw-insn", str(tmp_path / part)], check=True, capture_output=True,
                              text=True).stdout
        yield [line.split("//")[0].strip() for line in text.splitlines() if line.startswith("\t")]


def test_loads_to_lds_wait_for_m0(tmp_path):
    """A load from global memory to LDS takes its LDS address from M0 and needs one wait state after a scalar write
    of M0: the instruction before it writes something else, or is an s_nop."""
    loads, unsafe = 0, []
    for code in device_code(tmp_path):
        for before, now in zip(code, code[1:]):
            if re.match(r"(global|buffer|scratch)_load_(lds_|.*\blds\b)", now):
                loads += 1
                if re.match(r"s_\w+ m0\b", before):
                    unsafe.append((before, now))
    assert loads > 0
    assert not unsafe, f"{len(unsafe)} of {loads} loads follow the write of M0 at once: {unsafe[0]}"
