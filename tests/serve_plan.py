"""The launch plan of single-token attention, read from the built library without a GPU."""
from __future__ import annotations

import ctypes

import weight_only_int4_amd as w4


class Plan(ctypes.Structure):
    """struct DecodePlan of csrc/internal.hpp."""
    _fields_ = ([(f, ctypes.c_int) for f in ("group", "prefix")] + [(f, ctypes.c_bool) for f in ("wide", "direct")] +
                [(f, ctypes.c_int) for f in ("p_chunk", "p_splits", "p_tiles", "o_chunk", "o_splits", "o_tiles", "splits")] +
                [(f, ctypes.c_size_t) for f in ("rows", "stats_bytes", "bytes")])

    @property
    def form(self):
        """What the prefix, or without one all keys, go through: "direct", "wide", "prefix" (narrow) or "own" (narrow chunks)."""
        return "direct" if self.direct else "wide" if self.wide else "prefix" if self.prefix else "own"


def plan(B, n_q, n_kv, head, page, max_len, prefix=0):
    fn = getattr(w4.load_library(), "_ZN2w411plan_decodeEiiRK11w4_kv_cacheii")    # w4::plan_decode(int, int, const w4_kv_cache&, int, int)
    fn.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.POINTER(w4._KVCache), ctypes.c_int, ctypes.c_int]
    fn.restype = Plan
    return fn(B, n_q, ctypes.byref(w4._KVCache(None, None, 1, page, n_kv, head)), max_len, prefix)
