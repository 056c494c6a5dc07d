"""The library's own plan of a product, compiled from its sources for the host.

A test whose sizes stand for a way in which a product is cut asks here that they still are cut so."""
import ctypes
import functools
import os
import subprocess
import tempfile

from matrix_aware_optimizer_amd import build as _build

KINDS = ("direct", "narrow", "small", "large")
SOURCE = r"""
#include "tile.h"
extern "C" int tile_plan(int64_t m, int64_t n, int64_t steps, int mats, int batch, int whole, int rows_only, int a_rows, int64_t* out) {
  const muon::tile::Plan p = muon::tile::plan_product(m, n, steps, mats, batch, whole != 0, rows_only != 0, a_rows != 0);
  const int64_t tiles = muon::tile::ceil_div(m, 256) * muon::tile::ceil_div(n, 256 / mats) * batch;
  out[0] = p.kind; out[1] = p.parts; out[2] = tiles; out[3] = muon::tile::last_round_parts(tiles);
  return 0;
}
"""


@functools.lru_cache(maxsize=None)
def _library():
    with tempfile.TemporaryDirectory() as d:
        src, lib = os.path.join(d, "plan.hip"), os.path.join(d, "plan.so")
        with open(src, "w") as f:
            f.write(SOURCE)
        flags = [x for x in _build.compile_flags() if x.startswith(("-I", "-std", "-W"))]
        subprocess.run([_build.hipcc(), "--offload-host-only", "-O1", "-fPIC", "-shared", *flags, src, "-o", lib], check=True, capture_output=True)
        return ctypes.CDLL(lib)


def plan(m, n, steps, mats=1, batch=1, whole=True, rows_only=True, a_rows=True):
    """(kind, parts of the contraction, 256 x 256 tiles, parts of each tile of their last round)."""
    out = (ctypes.c_int64 * 4)()
    _library().tile_plan(*(ctypes.c_int64(v) for v in (m, n, steps)), mats, batch, whole, rows_only, a_rows, out)
    return KINDS[out[0]], out[1], out[2], out[3]


def int8(m, n, K, mats=1):
    return plan(m, n, -(-K // 64), mats)


def forward(t, f, d, whole=True):
    return plan(t, f, d // 32, 2, 1, whole)


def backward(t, f, d, whole=True):
    return plan(t, d, 2 * (f // 32), 1, 1, whole, rows_only=False)


def weights(t, f, d, whole=True):
    return plan(f, d, t // 32, 1, 2, whole, rows_only=False, a_rows=False)
