"""The launch plan of an MXFP4 product, read from the built library without a GPU."""
from __future__ import annotations

import ctypes
import random

import weight_only_int4_amd as w4


class _Stream(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int) for f in ("slices", "rows", "cols", "waves", "splits")]


class _Tile(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int) for f in ("tile", "splits", "stages")] + [("chain", ctypes.c_bool)]


class _Plan(ctypes.Structure):
    """struct MxPlan of csrc/internal.hpp."""
    _fields_ = [("use_tile", ctypes.c_bool), ("fits", ctypes.c_bool), ("stream", _Stream), ("tile", _Tile),
                ("workspace", ctypes.c_size_t)]


TILES = {16: ("256x192", "128x128", "128x64", "64x64"), 4: ("256x256", "256x192", "128x128", "128x64", "64x64")}


def plan(act, M, K, N):
    """("stream", slices, row tiles, channel tiles, split of K), ("tile", shape, split of K, chained, padded scales),
    or None where the shape is refused."""
    fn = getattr(w4.load_library(), "_ZN2w415plan_mxfp4_gemmEiiii")       # w4::plan_mxfp4_gemm(int, int, int, int)
    fn.argtypes, fn.restype = [ctypes.c_int] * 4, _Plan
    p = fn(act, M, K, N)
    if not p.fits:
        return None
    if not p.use_tile:
        return "stream", p.stream.slices, p.stream.rows, p.stream.cols, p.stream.splits
    blocks = K // 32
    return "tile", TILES[act][p.tile.tile], p.tile.splits, p.tile.chain, blocks % 4 != 0 or blocks < 16


def random_shapes(count, seed):
    """Shapes over the whole range of the products, sizes spread over their logarithm."""
    rng = random.Random(seed)

    def spread(lo, hi):
        return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))

    for _ in range(count):
        yield (rng.choice((16, 4)), rng.choice((spread(1, 70), spread(1, 4096), spread(1, 10 ** 6))),
               32 * spread(1, rng.choice((544, 65536))), spread(1, rng.choice((20000, 10 ** 7))))
