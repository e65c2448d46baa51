"""CPU oracle for the MXFP4 operators (4-bit microscaling floats).

TEST INFRASTRUCTURE ONLY, as w4a16_oracle: the plain statement of what the GPU path
computes, in NumPy fp64, sharing no code with the library.

Source: Open Compute Project, "OCP Microscaling Formats (MX) Specification v1.0", sections
5.2 (concrete formats: MXFP4 = 32 elements of e2m1 with one E8M0 scale) and 6.3
(conversion: the shared exponent is floor(log2 max|v|) minus the largest exponent of the
element type, elements rounded to nearest even and saturated).  Readings: the shared
exponent is clamped to E8M0's range, with byte 0 for a zero or fp32-subnormal maximum; a block with an
infinite or NaN value has byte 255 and codes 0; the sign of zero is kept.
"""
from __future__ import annotations

import numpy as np

BLOCK = 32
EMAX_ELEM = 2                                          # 6 = 1.5 * 2^2
MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def round_e2m1(y: np.ndarray) -> np.ndarray:
    """Magnitude codes 0..7 of |y|: the nearest magnitude, ties to the even code, 6 at most."""
    a = np.minimum(np.abs(np.asarray(y, dtype=np.float64)), 6.0)
    d = np.abs(a[..., None] - MAGNITUDES)
    low = np.argmin(d, axis=-1)                        # the lower code of a tie
    high = 7 - np.argmin(d[..., ::-1], axis=-1)        # the upper one
    return np.where(low % 2 == 0, low, high).astype(np.uint8)


def quantize(v: np.ndarray):
    """fp32 v [N][K] -> (codes uint8 [N][K] in 0..15, scale bytes uint8 [N][K/32])."""
    v = np.asarray(v, dtype=np.float32)
    n, k = v.shape
    if k % BLOCK:
        raise ValueError("K must be a multiple of 32")
    b = v.reshape(n, k // BLOCK, BLOCK).astype(np.float64)
    top = np.abs(b).max(axis=2)
    bad = ~np.isfinite(b).all(axis=2)
    safe = np.where(bad | (top < 2.0 ** -126), 1.0, top)
    exponent = np.frexp(safe)[1] - 1                   # floor(log2)
    byte = np.clip(exponent - EMAX_ELEM + 127, 0, 254)
    byte = np.where(top < 2.0 ** -126, 0, byte)
    byte = np.where(bad, 255, byte).astype(np.uint8)
    with np.errstate(invalid="ignore"):
        y = b / np.ldexp(1.0, byte.astype(np.int64) - 127)[..., None]
    codes = round_e2m1(np.where(bad[..., None], 0.0, y)) | (np.signbit(b).astype(np.uint8) << 3)
    codes = np.where(bad[..., None], 0, codes).astype(np.uint8)
    return codes.reshape(n, k), byte


def pack(codes: np.ndarray) -> np.ndarray:
    """codes uint8 [..., K] -> uint32 words [..., K/8], the first code in the lowest bits."""
    c = np.asarray(codes, dtype=np.uint32).reshape(*codes.shape[:-1], -1, 8)
    return (c << (4 * np.arange(8, dtype=np.uint32))).sum(axis=-1, dtype=np.uint64).astype(np.uint32)


def unpack(words: np.ndarray) -> np.ndarray:
    w = np.asarray(words, dtype=np.uint32)
    c = (w[..., None] >> (4 * np.arange(8, dtype=np.uint32))) & np.uint32(15)
    return c.reshape(*w.shape[:-1], -1).astype(np.uint8)


def dequantize(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """fp64 values of codes uint8 [N][K] with scale bytes [N][K/32]; NaN where the byte is 255."""
    n, k = codes.shape
    sign = np.where(codes & 8, -1.0, 1.0)
    v = (sign * MAGNITUDES[codes & 7]).reshape(n, k // BLOCK, BLOCK)
    scale = np.ldexp(1.0, scales.astype(np.int64) - 127)
    scale = np.where(scales == 255, np.nan, scale)
    return (v * scale[..., None]).reshape(n, k)


def product_bound(x: np.ndarray, w: np.ndarray):
    """(x w^T in fp64, the largest distance a kernel's bf16 output may have from it).

    Products of the operands are exact in fp32, so what is left is the fp32 accumulation --
    at most K - 1 additions, each off by at most 2^-23 of a partial sum (truncation counted,
    twice the half step of rounding to nearest), a partial sum being at most sum |x||w| --
    and one rounding to bf16: half a step, 2^-8 of the value, or 2^-134 where that is
    subnormal."""
    ref = x @ w.T
    acc = x.shape[1] * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T)
    return ref, acc + 2.0 ** -8 * (np.abs(ref) + acc) + 2.0 ** -134
