"""The serving operators without a GPU: the oracle against scalar restatements and closed forms,
and the entry points' refusals."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest
import torch

import weight_only_int4_amd as w4
from oracle import serve_oracle as SO

P = ctypes.c_void_p
A = P(0x10000)        # a 16-byte aligned fake device address (never dereferenced)
MIS = P(0x10004)


@pytest.fixture(scope="module")
def lib():
    return w4.load_library()


# ---------------------------------------------------------------- oracle pins

def _bf(rng, *shape):
    return SO.bf16(rng.standard_normal(shape))


def test_bf16_rounds_to_even_and_keeps_specials():
    x = np.array([1.0, 1 + 2 ** -8, 1 + 3 * 2 ** -8, np.inf, -np.inf, np.nan], np.float32)
    y = SO.bf16(x)
    assert y[:5].tolist() == [1.0, 1.0, 1 + 2 ** -6, math.inf, -math.inf] and math.isnan(y[5])


def test_norm_scalar_restatement():
    rng = np.random.default_rng(1)
    x, res, w = _bf(rng, 3, 256), _bf(rng, 3, 256), _bf(rng, 256)
    h = SO.norm_sum(x, res)
    y, (codes, sx, xsum) = SO.rmsnorm(h, w, 1e-5), SO.rmsnorm_int8(h, w, 1e-5)
    for m in range(3):
        r = 1 / math.sqrt(sum(float(a) ** 2 for a in h[m]) / 256 + 1e-5)
        want = [float(a) * r * float(b) for a, b in zip(h[m], w)]
        assert np.allclose(y[m], want, rtol=1e-13)
        top = max(abs(a) for a in want)
        assert abs(sx[m] - top / 127) <= 1e-6 * sx[m]
        # a code times the scale lies within half a step of the value
        assert np.max(np.abs(codes[m] * sx[m] - want)) <= sx[m] * (0.5 + 1e-4)
        assert abs(codes[m]).max() == 127
        assert xsum[m].tolist() == [int(codes[m, :128].astype(int).sum()), int(codes[m, 128:].astype(int).sum())]


def test_norm_int8_special_rows():
    h = np.zeros((3, 128), np.float32)
    h[1, 5], h[2, 7] = np.inf, np.nan
    codes, sx, xsum = SO.rmsnorm_int8(h, np.ones(128, np.float32), 1.0)
    assert not codes.any() and not xsum.any() and sx[0] == 1.0 and np.isnan(sx[1:]).all()


def test_rotation_keeps_lengths_and_depends_on_differences():
    rng = np.random.default_rng(2)
    cs, sn = (a.astype(np.float32) for a in SO.rope_table(50, 64, 1e4))
    assert (cs[0] == 1).all() and (sn[0] == 0).all()
    x = _bf(rng, 50, 2, 64)
    y = SO.rotate(x, cs, sn)
    assert np.array_equal(y[0], x[0])
    pairs = lambda a: a[..., :32].astype(float) ** 2 + a[..., 32:].astype(float) ** 2  # noqa: E731
    assert np.allclose(pairs(y), pairs(x), rtol=2 ** -6, atol=1e-6)
    a, b = _bf(rng, 1, 1, 64), _bf(rng, 1, 1, 64)
    dot = [float((SO.rotate(a, cs[p:p + 1], sn[p:p + 1]) * SO.rotate(b, cs[p + 7:p + 8], sn[p + 7:p + 8])).sum()) for p in (0, 11, 40)]
    assert max(dot) - min(dot) <= 64 * 2 ** -6


def test_attention_scalar_restatement_and_special_cases():
    rng = np.random.default_rng(3)
    q, k, v = _bf(rng, 9, 4, 64), _bf(rng, 9, 2, 64), _bf(rng, 9, 2, 64)
    got = SO.prompt_attention(q, k, v, [0, 4, 4, 9], 0.125)
    assert len(got) == 9 * 4
    for (t, h), a in got.items():
        first = 0 if t < 4 else 4
        s = [0.125 * sum(float(x) * float(y) for x, y in zip(q[t, h], k[j, h // 2])) for j in range(first, t + 1)]
        e = [math.exp(x - max(s)) for x in s]
        want = [sum(p * float(v[first + j, h // 2, d]) for j, p in enumerate(e)) / sum(e) for d in range(64)]
        assert np.allclose(a.o, want, rtol=1e-12, atol=1e-14)
    assert np.array_equal(got[4, 1].o, v[4, 0])                     # a first token returns its value
    # the same keys through pages, two of three shared
    kc, vc = np.zeros((5, 2, 16, 64), np.float32), np.zeros((5, 2, 16, 64), np.float32)
    kk, vv = _bf(rng, 40, 2, 64), _bf(rng, 40, 2, 64)
    for p in range(40):
        kc[[4, 0, 2][p // 16], :, p % 16], vc[[4, 0, 2][p // 16], :, p % 16] = kk[p], vv[p]
    table = np.array([[4, 0, -1], [99, -7, 2]])
    out = SO.decode_attention(q[:2], kc, vc, [32, 40], table, 32, 0.125)
    for b, n in ((0, 32), (1, 40)):
        for h in range(4):
            assert np.allclose(out[b, h].o, SO.Attention(q[b, h], kk[:n, h // 2], vv[:n, h // 2], 0.125).o)
    # a key without a page is left out, an empty sequence is zero
    out = SO.decode_attention(q[:2], kc, vc, [40, 0], table, 0, 0.125)
    assert np.allclose(out[0, 0].o, SO.Attention(q[0, 0], kk[:32, 0], vv[:32, 0], 0.125).o)
    assert not out[1, 3].o.any()


def test_append_places_tokens():
    rng = np.random.default_rng(4)
    q, k, v = _bf(rng, 6, 2, 64), _bf(rng, 6, 1, 64), _bf(rng, 6, 1, 64)
    cs, sn = (a.astype(np.float32) for a in SO.rope_table(40, 64, 1e6))
    kc, vc = np.full((3, 1, 16, 64), 9, np.float32), np.full((3, 1, 16, 64), 9, np.float32)
    qo, ko = np.full_like(q, 7), np.full_like(k, 7)
    # 2 tokens that end at 18 (page 1 of the table is page 0), none, 3 that begin before 0; row 5 behind the last
    SO.append(q, k, v, cs, sn, kc, vc, [18, 5, 2], np.array([[2, 0], [0, 0], [1, 0]]), [0, 2, 2, 5], qo, ko)
    assert np.array_equal(vc[0, :, 0], v[0]) and np.array_equal(vc[0, :, 1], v[1])
    assert (qo[2] == 7).all() and (qo[5] == 7).all()               # position -1, and no sequence
    assert np.array_equal(qo[3], q[3]) and np.array_equal(vc[1, :, 0], v[3]) and np.array_equal(vc[1, :, 1], v[4])
    assert np.array_equal(kc[0, :, 0], SO.rotate(k[:1], cs[16:17], sn[16:17])[0])
    assert (kc != 9).any(axis=(1, 3)).sum() == 4


def test_what_device_arrays_say_is_held_in_range(tmp_path):
    """The kernels' own functions for offsets, lengths, positions and page numbers, compiled for the host."""
    here = os.path.dirname(os.path.abspath(__file__))
    exe = str(tmp_path / "held_check")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-o", exe, os.path.join(here, "held_check.cpp")], check=True)
    res = subprocess.run([exe], capture_output=True, text=True)
    assert res.returncode == 0, res.stdout


# ---------------------------------------------------------------- refusals of the C entry points

def test_norm_refusals(lib):
    f = lambda X=A, r=A, T=4, H=256, w=A, eps=1e-6, h=A, Y=A: lib.w4_rmsnorm(X, r, T, H, w, eps, h, Y, None)  # noqa: E731
    g = lambda X=A, r=A, T=4, H=256, w=A, eps=1e-6, h=A, q=A, s=A, x=A: lib.w4a8_rmsnorm(X, r, T, H, w, eps, h, q, s, x, None)  # noqa: E731
    for fn in (f, g):
        for bad in (0, -8, 100, 65536 + 128):
            assert fn(H=bad) == -2
        assert fn(T=-1) == -2 and fn(T=2 ** 31 - 1) == -2
        for eps in (-1e-6, math.nan, math.inf):
            assert fn(eps=eps) == -7
        assert fn(X=None) == -1 and fn(w=None) == -1
        assert fn(r=None) == -1 and fn(h=None) == -1               # a residual and its sum go together
        for name in ("X", "r", "w", "h"):
            assert fn(**{name: MIS}) == -3
        assert fn(T=0, X=None, r=None, w=None, h=None) == 0
    assert f(Y=None) == -1 and f(Y=MIS) == -3
    assert g(H=136) == -2
    for name in "qsx":
        assert g(**{name: None}) == -1 and g(**{name: MIS}) == -3


def test_rope_table_refusals(lib):
    f = lib.w4_rope_table
    assert f(16, 96, 1e6, A, A, None) == -4
    assert f(-1, 64, 1e6, A, A, None) == -2 and f(2 ** 31 - 1, 128, 1e6, A, A, None) == -2
    for base in (0.0, -1.0, math.inf, math.nan):
        assert f(16, 64, base, A, A, None) == -7
    assert f(16, 64, 1e6, None, A, None) == -1 and f(16, 64, 1e6, A, MIS, None) == -3
    assert f(0, 64, 1e6, None, None, None) == 0


def _cache(k=0x10000, v=0x20000, pages=9, page_size=16, n_kv=2, head=64):
    return w4._KVCache(k, v, pages, page_size, n_kv, head)


def _append(lib, cache=None, **kw):
    a = dict(Q=A, qs=256, K=A, ks=128, V=A, vs=128, T=3, n_q=4, off=A, lens=A, B=2, table=A, width=5, cs=A, sn=A, P=100, qo=A, ko=A)
    a.update(kw)
    c = _cache() if cache is None else cache
    return lib.w4_kv_append(a["Q"], a["qs"], a["K"], a["ks"], a["V"], a["vs"], a["T"], a["n_q"], a["off"], a["lens"], a["B"], a["table"],
                            a["width"], a["cs"], a["sn"], a["P"], ctypes.byref(c), a["qo"], a["ko"], None)


def test_append_refusals(lib):
    assert lib.w4_kv_append(A, 256, A, 128, A, 128, 3, 4, A, A, 2, A, 5, A, A, 100, None, A, A, None) == -1
    for c in (dict(head=96), dict(page_size=24), dict(page_size=8), dict(page_size=512)):
        assert _append(lib, _cache(**c)) == -4
    for c in (dict(n_kv=0), dict(n_kv=3), dict(pages=-1)):
        assert _append(lib, _cache(**c)) == -2
    for kw in (dict(T=-1), dict(B=-1), dict(width=-1), dict(P=-1), dict(n_q=0), dict(n_q=5), dict(off=None), dict(qs=248), dict(qs=260),
               dict(ks=120), dict(vs=64), dict(T=2 ** 31 - 1), dict(ks=-128)):
        assert _append(lib, **kw) == -2, kw
    for name in ("Q", "K", "V", "lens", "table", "cs", "sn", "qo"):
        assert _append(lib, **{name: None}) == -1, name
        assert _append(lib, **{name: MIS}) == -3, name
    assert _append(lib, ko=MIS) == -3 and _append(lib, off=MIS) == -3
    assert _append(lib, _cache(k=None)) == -1 and _append(lib, _cache(v=0x20008)) == -3
    assert _append(lib, T=0, Q=None) == 0 and _append(lib, B=0, T=0, off=None) == 0


def _prompt(lib, **kw):
    a = dict(Q=A, qs=512, K=A, ks=256, V=A, vs=256, T=9, n_q=4, n_kv=2, head=128, off=A, B=2, scale=0.1, O=A)
    a.update(kw)
    size = ctypes.c_size_t(0)
    lib.w4_prompt_attention(None, 0, None, 0, None, 0, a["T"], a["n_q"], a["n_kv"], a["head"], None, a["B"], 0.0, None, None,
                            ctypes.byref(size), None)
    ws = (A, ctypes.byref(size)) if size.value else (None, None)
    return lib.w4_prompt_attention(a["Q"], a["qs"], a["K"], a["ks"], a["V"], a["vs"], a["T"], a["n_q"], a["n_kv"], a["head"], a["off"],
                                   a["B"], a["scale"], a["O"], *ws, None)


def test_prompt_refusals(lib):
    assert _prompt(lib, head=80) == -4
    for kw in (dict(T=-1), dict(B=-1), dict(n_q=0), dict(n_kv=0), dict(n_q=5), dict(qs=511), dict(qs=504), dict(ks=128), dict(vs=0),
               dict(T=2 ** 31 - 1, n_q=64, qs=64 * 128)):
        assert _prompt(lib, **kw) == -2, kw
    for scale in (0.0, -1.0, math.nan, math.inf):
        assert _prompt(lib, scale=scale) == -7
    for name in ("Q", "K", "V", "off", "O"):
        assert _prompt(lib, **{name: None}) == -1, name
        assert _prompt(lib, **{name: MIS}) == -3, name
    assert _prompt(lib, T=0, Q=None) == 0 and _prompt(lib, B=0) == 0


def _decode(lib, cache=None, ws=None, **kw):
    a = dict(Q=A, qs=256, B=3, n_q=4, lens=A, table=A, width=5, max_len=80, prefix=32, scale=0.1, O=A)
    a.update(kw)
    c = _cache() if cache is None else cache
    if ws is None:
        size = ctypes.c_size_t(0)
        lib.w4_decode_attention(None, 0, a["B"], a["n_q"], ctypes.byref(c), None, None, 0, a["max_len"], a["prefix"], 0.0, None, None,
                                ctypes.byref(size), None)
        ws = (A, ctypes.byref(size)) if size.value else (None, None)
    return lib.w4_decode_attention(a["Q"], a["qs"], a["B"], a["n_q"], ctypes.byref(c), a["lens"], a["table"], a["width"], a["max_len"],
                                   a["prefix"], a["scale"], a["O"], *ws, None)


def test_decode_refusals(lib):
    assert lib.w4_decode_attention(A, 256, 3, 4, None, A, A, 5, 80, 32, 0.1, A, None, None, None) == -1
    assert _decode(lib, _cache(head=32)) == -4 and _decode(lib, _cache(page_size=17)) == -4
    for kw in (dict(B=-1), dict(n_q=3), dict(max_len=-1), dict(max_len=81), dict(prefix=-16), dict(prefix=24), dict(prefix=96),
               dict(width=-1), dict(qs=128), dict(qs=260), dict(width=2 ** 31 - 1, max_len=2 ** 31 - 1),
               dict(width=2 ** 31 - 1, max_len=2 ** 30 + 1), dict(B=2 ** 31 - 1), dict(B=2 ** 23, width=2 ** 20, max_len=2 ** 23),
               dict(width=2 ** 27, max_len=2 ** 30, prefix=2 ** 30 + 16)):
        assert _decode(lib, **kw) == -2, kw
    for scale in (0.0, -1.0, math.nan, math.inf):
        assert _decode(lib, scale=scale) == -7
    for name in ("Q", "lens", "table", "O"):
        assert _decode(lib, **{name: None}) == -1, name
        assert _decode(lib, **{name: MIS}) == -3, name
    assert _decode(lib, _cache(v=None)) == -1 and _decode(lib, _cache(k=0x10008)) == -3
    assert _decode(lib, B=0, Q=None) == 0


def test_decode_workspace_sizes(lib):
    """The size query over the range of its arguments: monotonous plans, no wrap-around, and the same for the same call."""
    def size(B, n_q, max_len, prefix, **kw):
        c, out = _cache(**kw), ctypes.c_size_t(0)
        rc = lib.w4_decode_attention(None, 0, B, n_q, ctypes.byref(c), None, None, 0, max_len, prefix, 0.0, None, None, ctypes.byref(out), None)
        return rc, out.value
    assert size(1, 4, 100, 0) == (0, 0) and size(0, 4, 100, 32) == (0, 0)
    for B in (1, 2, 3, 16, 64, 65, 200, 1000):
        for max_len in (0, 1, 127, 500, 1025, 5000, 70000):
            for prefix in (0, 16, 512, 4096):
                for heads in ((1, 1), (16, 8), (64, 4), (48, 1)):
                    rc, n = size(B, heads[0], max_len, prefix, n_kv=heads[1], head=128)
                    rows = B * heads[0]
                    assert rc == 0 and n == size(B, heads[0], max_len, prefix, n_kv=heads[1], head=128)[1]
                    # splits x rows x (m, l and 128 sums), the first part rounded up to 256 bytes
                    assert n == 0 or any(n == -(-k * rows * 8 // 256) * 256 + k * rows * 512 for k in range(1, 2000))
                    if B > 1 and prefix and max_len:
                        assert n > 0
    rc, n = size(1, 1, 2 ** 30, 0, n_kv=1)
    assert rc == 0 and n >= 2 ** 20 * (8 + 4 * 64)


def test_binding_refusals():
    """What the binding checks before the library is asked (CPU tensors are refused)."""
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    w = torch.zeros(256, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        w4.rmsnorm(x, w)
    with pytest.raises(TypeError):
        w4.w4a8_rmsnorm(x.float(), w)
    with pytest.raises(ValueError):
        w4.rope_table(-1, 128)
    with pytest.raises(ValueError):
        w4.rope_table(4, 128, device="cpu")
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    ints = torch.zeros(5, dtype=torch.int32)
    cache = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16)
    for call in (lambda: w4.prompt_attention(q, q, q, ints), lambda: w4.decode_attention(q, cache, cache, ints[:4], ints.reshape(5, 1)),
                 lambda: w4.kv_append(q, q, q, x.float(), x.float(), cache, cache, ints[:4], ints.reshape(5, 1))):
        with pytest.raises(ValueError):
            call()
