"""Plain CPU oracle of the serving operators (test infrastructure only): norm with residual and
int8 output, rotary append to a paged cache, causal attention of packed prompts, attention of
single tokens over the cache.  NumPy; fp32 steps where the definition is in fp32 (codes,
rotation), fp64 elsewhere.  bf16 data as fp32 arrays that hold bf16 values."""
from __future__ import annotations

import numpy as np

from oracle.w4a16_oracle import bf16_to_f32, f32_to_bf16


def bf16(x):
    """fp32 values rounded to bf16, to nearest even (NaN and infinities kept)."""
    x = np.asarray(x, np.float32)
    return np.where(np.isfinite(x), bf16_to_f32(f32_to_bf16(np.where(np.isfinite(x), x, 0).astype(np.float32))), x).astype(np.float32)


def norm_sum(x, residual):
    return x if residual is None else bf16(x + residual)


def rmsnorm(h, weight, eps):
    """fp64 [T][H]."""
    h = h.astype(np.float64)
    return h / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps) * weight.astype(np.float64)


def rmsnorm_int8(h, weight, eps):
    """(codes int8, sx fp64, xsum int32)."""
    with np.errstate(all="ignore"):
        v = (h * weight).astype(np.float32)
        top = np.abs(v).max(axis=1)
        bad = ~np.isfinite(v).all(axis=1)
        t = (top * (np.float32(1) / np.float32(127))).astype(np.float32)
        t = np.where(t == 0, np.float32(1), t)
        codes = np.clip(np.rint(v / t[:, None]), -127, 127)
        h64 = h.astype(np.float64)
        sx = t.astype(np.float64) / np.sqrt((h64 * h64).mean(axis=1) + eps)
    codes[bad], sx[bad] = 0, np.nan
    return codes.astype(np.int8), sx, codes.reshape(len(codes), -1, 128).sum(axis=2).astype(np.int32)


def rope_table(positions, head, base):
    angle = np.arange(positions)[:, None] * float(base) ** (-2.0 * np.arange(head // 2) / head)
    return np.cos(angle), np.sin(angle)


def rotate(x, c, s):
    """x [n][heads][head] fp32, c and s [n][head/2] fp32: every product and sum rounded to fp32, then bf16."""
    half = x.shape[2] // 2
    a, b, c, s = x[..., :half], x[..., half:], c[:, None], s[:, None]
    return bf16(np.concatenate((a * c - b * s, b * c + a * s), axis=2))


def append(q, k, v, cs, sn, k_cache, v_cache, lens, table, offsets, q_out, k_out):
    """Writes q_out, k_out and the caches in place, token by token."""
    page_size, pages = k_cache.shape[2], k_cache.shape[0]
    for b in range(len(lens)):
        n = offsets[b + 1] - offsets[b]
        for i in range(n):
            t, p = offsets[b] + i, int(lens[b]) - n + i
            if p < 0 or p >= len(cs):
                continue
            q_out[t] = rotate(q[t:t + 1], cs[p:p + 1], sn[p:p + 1])[0]
            k_out[t] = rotate(k[t:t + 1], cs[p:p + 1], sn[p:p + 1])[0]
            entry = p // page_size
            page = int(table[b, entry]) if entry < table.shape[1] else -1
            if 0 <= page < pages:
                k_cache[page, :, p % page_size] = k_out[t]
                v_cache[page, :, p % page_size] = v[t]


class Attention:
    """One query's result o [head] with what its error bound needs: spread = sum p |v| / sum p,
    noise = sqrt(sum p^2 v^2) / sum p, and the largest sum of |q k| times scale."""

    def __init__(self, q, k, v, scale):
        q, k, v = q.astype(np.float64), k.astype(np.float64), v.astype(np.float64)
        if len(k) == 0:
            self.o = self.spread = self.noise = np.zeros(len(q))
            self.reach = 0.0
            return
        s = scale * (k @ q)
        p = np.exp(s - s.max())
        p /= p.sum()
        self.o, self.spread, self.noise = p @ v, p @ np.abs(v), np.sqrt((p * p) @ (v * v))
        self.reach = scale * float((np.abs(k) @ np.abs(q)).max())


def prompt_attention(q, k, v, offsets, scale):
    """{(token, head): Attention} of every token of every sequence."""
    group = q.shape[1] // k.shape[1]
    return {(t, h): Attention(q[t, h], k[a:t + 1, h // group], v[a:t + 1, h // group], scale)
            for a, b in zip(offsets[:-1], offsets[1:]) for t in range(a, b) for h in range(q.shape[1])}


def decode_attention(q, k_cache, v_cache, lens, table, prefix_len, scale):
    """{(sequence, head): Attention}; keys on pages outside the cache are left out."""
    page_size, pages = k_cache.shape[2], k_cache.shape[0]
    group = q.shape[1] // k_cache.shape[1]
    out = {}
    for b in range(len(lens)):
        p = np.arange(max(int(lens[b]), 0))
        page = table[np.where(p < prefix_len, 0, b), p // page_size]
        kept = (page >= 0) & (page < pages)
        page, slot = page[kept], p[kept] % page_size
        for h in range(q.shape[1]):
            out[b, h] = Attention(q[b, h], k_cache[page, h // group, slot], v_cache[page, h // group, slot], scale)
    return out
