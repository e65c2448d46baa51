"""The serving operators on the GPU against the CPU oracle and plain 64-bit attention.

Tolerances.  Sums h, codes, code sums, rotated values and cache slots: bit for bit (fp32 steps
without reordering).  sx: its fp32 sum of H squares runs in chains of at most H / 64 additions and
a tree, each addition off by 2^-24, halved by the root, and a few single roundings.  y: that and
half a step of bf16 (2^-8).  Attention, per element, S = sum p |v| / sum p:
  scores: head fp32 additions of exact products, off by 2^-23 of sum |q k| each (truncation
  counted), the scale and the exponent's argument a few roundings more: p is off by
  e = reach (head + 8) 2^-23 + 2^-20 relative, reach = scale max sum |q k|; p is rounded to bf16
  (2^-8); n additions in fp32, 2^-23 each, above and below the fraction; so
  |o - o'| <= (2^-8 + 2 e + 2 n 2^-23) S + 2^-8 |o|.
The roundings of p and o are independent, so over many elements the root mean square is held to
that of 2^-8 sqrt(sum p^2 v^2) / sum p and 2^-8 o (a uniform rounding has 0.58 of it), plus the terms in e and n."""
import math

import numpy as np
import pytest
import torch

import weight_only_int4_amd as w4
import workloads as wl
from oracle import serve_oracle as SO
from oracle import w4a16_oracle as O
from tests.gpu_util import gpu_available, say

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs an MI355X GPU")]

BF = torch.bfloat16
NAN, INF = float("nan"), float("inf")


def gpu(a, dtype=BF):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda").to(dtype)


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def host(t):
    return t.detach().float().cpu().numpy()


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


def normal(rng, *shape):
    return SO.bf16(rng.standard_normal(shape))


# ---------------------------------------------------------------- norm

def _check_norm(x, res, w, eps, y=None, h=None, int8=None):
    """Compares what was given of the outputs with the oracle."""
    H = x.shape[1]
    hs = SO.norm_sum(x, res)
    rel = ((H / 64 + 16) / 2 + 6) * 2.0 ** -24
    if h is not None:
        assert np.array_equal(host(h), hs, equal_nan=True)
    if y is not None:
        want = SO.rmsnorm(hs, w, eps)
        fine = np.isfinite(want)
        got = host(y).astype(np.float64)
        assert np.array_equal(fine, np.isfinite(got))
        off = np.abs(got - want)[fine]
        assert (off <= (2.0 ** -8 + 4 * rel) * np.abs(want)[fine] + 1e-40).all(), off.max()
    if int8 is not None:
        codes, sx, xsum = SO.rmsnorm_int8(hs, w, eps)
        assert np.array_equal(int8[0].cpu().numpy(), codes)
        assert np.array_equal(int8[2].cpu().numpy(), xsum)
        got = int8[1].cpu().numpy().astype(np.float64)
        assert np.array_equal(np.isnan(got), np.isnan(sx))
        fine = ~np.isnan(sx)
        assert (np.abs(got - sx)[fine] <= rel * sx[fine]).all()


NORM_SIZES = [(1, 128), (3, 256), (37, 2048), (5, 2176), (16, 5120), (2, 6144), (130, 896), (3, 17408), (1, 32768), (2, 65536), (1025, 128)]


@pytest.mark.parametrize("T,H", NORM_SIZES + [(1, 8), (7, 136), (4, 2056), (300, 520), (2, 16392), (1, 65528)])
@pytest.mark.parametrize("with_res", [False, True])
def test_rmsnorm(T, H, with_res):
    say("rmsnorm", T, H, with_res)
    rng = np.random.default_rng(T * 7 + H)
    x, res, w = normal(rng, T, H), normal(rng, T, H) if with_res else None, SO.bf16(1 + 0.2 * rng.standard_normal(H))
    x[:, rng.integers(0, H, max(1, H // 100))] *= 32
    y, h = w4.rmsnorm(gpu(x), gpu(w), None if res is None else gpu(res), 1e-6)
    assert (h is None) == (res is None)
    _check_norm(x, res, w, 1e-6, y, h)
    y2, _ = w4.rmsnorm(gpu(x), gpu(w), None if res is None else gpu(res), 1e-6)
    assert same_bits(y, y2)


@pytest.mark.parametrize("T,H", NORM_SIZES)
@pytest.mark.parametrize("with_res", [False, True])
def test_w4a8_rmsnorm(T, H, with_res):
    say("w4a8_rmsnorm", T, H, with_res)
    rng = np.random.default_rng(T * 11 + H)
    x, res, w = normal(rng, T, H), normal(rng, T, H) if with_res else None, SO.bf16(1 + 0.2 * rng.standard_normal(H))
    x[:, rng.integers(0, H, max(1, H // 100))] *= 32
    *int8, h = w4.w4a8_rmsnorm(gpu(x), gpu(w), None if res is None else gpu(res), 1e-5)
    _check_norm(x, res, w, 1e-5, None, h, int8)


def test_w4a8_rmsnorm_ties_and_scales():
    """Quotients on and next to half-integers, at every magnitude of bf16."""
    rng = np.random.default_rng(8)
    x = np.zeros((254, 256), np.float32)
    for i, e in enumerate(range(-126, 128)):
        x[i] = SO.bf16(rng.integers(-254, 255, 256) / 2.0 * 2.0 ** min(e, 120) * 2.0 ** -7)
        x[i, 0] = 127 * 2.0 ** min(e, 120) * 2.0 ** -7          # t is a power of two
    x = SO.bf16(x)
    w = np.ones(256, np.float32)
    *int8, _ = w4.w4a8_rmsnorm(gpu(x), gpu(w), None, 0.0)
    codes, _, xsum = SO.rmsnorm_int8(x, w, 0.0)
    assert np.array_equal(int8[0].cpu().numpy(), codes) and np.array_equal(int8[2].cpu().numpy(), xsum)


def test_w4a8_rmsnorm_quotients_next_to_halves():
    """Two million quotients of steps that are no powers of two: some hundred of them lie within 2^-14 of a half, where
    a product with the step's reciprocal could round the other way."""
    rng = np.random.default_rng(81)
    x = normal(rng, 2048, 1024) * np.float32(2.0) ** rng.integers(-90, 90, (2048, 1)).astype(np.float32)
    x, w = SO.bf16(x), SO.bf16(1 + 0.5 * rng.standard_normal(1024))
    codes, _, xsum = SO.rmsnorm_int8(x, w, 0.0)
    *int8, _ = w4.w4a8_rmsnorm(gpu(x), gpu(w), None, 0.0)
    assert np.array_equal(int8[0].cpu().numpy(), codes) and np.array_equal(int8[2].cpu().numpy(), xsum)


def test_w4a8_rmsnorm_smallest_values():
    """Products that are subnormal or underflow, and a step that underflows: the codes are the definition's."""
    rng = np.random.default_rng(18)
    x = SO.bf16(rng.integers(-255, 256, (6, 256)) * 2.0 ** -133)
    w = SO.bf16(2.0 ** rng.integers(-20, 1, 256))
    x[1], x[2] = SO.bf16(np.full(256, 2.0 ** -133)), 0
    x[3, 1:] = 0
    w[:8] = 2.0 ** -16
    *int8, _ = w4.w4a8_rmsnorm(gpu(x), gpu(w), None, 1e-6)
    _check_norm(x, None, w, 1e-6, None, None, int8)
    w[:] = 2.0 ** -16                                            # every |v| below 127 of the smallest number
    *int8, _ = w4.w4a8_rmsnorm(gpu(x[1:4] * 0 + x[1]), gpu(w), None, 1e-6)
    _check_norm(x[1:4] * 0 + x[1], None, w, 1e-6, None, None, int8)
    assert not int8[0].any() and (int8[1] > 0).all()


@pytest.mark.parametrize("H", [128, 2048, 8192])
def test_norm_special_rows(H):
    """Zero rows, and rows with infinities and NaN: the latter must not reach their neighbours."""
    rng = np.random.default_rng(H)
    x, w = normal(rng, 9, H), SO.bf16(1 + 0.2 * rng.standard_normal(H))
    x[1] = 0
    x[3, 5], x[5, H - 1], x[7, 64] = INF, -INF, NAN
    *int8, _ = w4.w4a8_rmsnorm(gpu(x), gpu(w), None, 1e-6)
    _check_norm(x, None, w, 1e-6, None, None, int8)
    y, _ = w4.rmsnorm(gpu(x), gpu(w), None, 1e-6)
    plain = [0, 1, 2, 4, 6, 8]
    _check_norm(x[plain], None, w, 1e-6, y[plain])
    assert torch.isnan(y[3]).any() and torch.isnan(y[5]).any() and torch.isnan(y[7]).all()
    wz = w.copy()
    wz[:] = 0
    *int8, _ = w4.w4a8_rmsnorm(gpu(x), gpu(wz), None, 1e-6)      # inf * 0 is NaN: the row's codes are 0
    _check_norm(x, None, wz, 1e-6, None, None, int8)


def test_norm_in_place_and_rows_behind():
    rng = np.random.default_rng(3)
    x, res, w = normal(rng, 6, 2048), normal(rng, 6, 2048), normal(rng, 2048)
    for target in ("x", "res"):
        gx, gr = gpu(x), gpu(res)
        y = torch.full((8, 2048), 7.0, dtype=BF, device="cuda")
        out, h = w4.rmsnorm(gx, gpu(w), gr, 1e-6, Y=y[:6], H=gx if target == "x" else gr)
        _check_norm(x, res, w, 1e-6, out, h)
        assert (y[6:] == 7).all() and h.data_ptr() == (gx if target == "x" else gr).data_ptr()
        gx, gr = gpu(x), gpu(res)
        *int8, h = w4.w4a8_rmsnorm(gx, gpu(w), gr, 1e-6, H=gx if target == "x" else gr)
        _check_norm(x, res, w, 1e-6, None, h, int8)
    gx = gpu(x)
    out, _ = w4.rmsnorm(gx, gpu(w), None, 1e-6, Y=gx)
    _check_norm(x, None, w, 1e-6, gx)
    empty = torch.empty(0, 2048, dtype=BF, device="cuda")
    assert w4.rmsnorm(empty, gpu(w))[0].shape == (0, 2048)


def test_norm_past_32_bit_offsets():
    T, H = 40000, 65536                                          # 2.6e9 elements
    x = torch.zeros(T, H, dtype=BF, device="cuda")
    rng = np.random.default_rng(5)
    rows = [0, 32767, 32768, T - 1]
    part, w = normal(rng, 4, H), normal(rng, H)
    x[rows] = gpu(part)
    y, _ = w4.rmsnorm(x, gpu(w), None, 1e-6, Y=x)
    _check_norm(part, None, w, 1e-6, y[rows])
    assert not y[1].any()


# ---------------------------------------------------------------- rope table and append

@pytest.mark.parametrize("positions,head,base", [(1, 64, 1e4), (5000, 128, 1e6), (131072, 64, 5e5)])
def test_rope_table(positions, head, base):
    cs, sn = w4.rope_table(positions, head, base)
    c, s = SO.rope_table(positions, head, base)
    tol = 2.0 ** -24 + positions * 2.0 ** -50
    assert np.abs(cs.cpu().numpy() - c).max() <= tol and np.abs(sn.cpu().numpy() - s).max() <= tol


def _append_case(rng, new, before, n_q, n_kv, head, page, fused=True, positions=None, spare=3):
    lens = [a + b for a, b in zip(new, before)]
    T = sum(new) + spare
    qkv = normal(rng, T, n_q + 2 * n_kv, head)
    q, k, v = qkv[:, :n_q], qkv[:, n_q:n_q + n_kv], qkv[:, n_q + n_kv:]
    width = max(1, max(-(-max(n, 0) // page) for n in lens))
    pages = len(new) * width + 2
    table = rng.permutation(pages)[:len(new) * width].reshape(len(new), width).astype(np.int32)
    P = max(lens) if positions is None else positions
    cs, sn = (a.astype(np.float32) for a in SO.rope_table(P, head, 1e6))
    kc, vc = normal(rng, pages, n_kv, page, head), normal(rng, pages, n_kv, page, head)
    offsets = [0]
    for n in new:
        offsets.append(offsets[-1] + n)
    return qkv, q, k, v, lens, table, cs, sn, kc, vc, offsets


def _run_append(case, use_offsets=True, with_k=True):
    qkv, q, k, v, lens, table, cs, sn, kc, vc, offsets = case
    g = gpu(qkv)
    n_q, n_kv = q.shape[1], k.shape[1]
    gq, gk, gv = g[:, :n_q], g[:, n_q:n_q + n_kv], g[:, n_q + n_kv:]
    gkc, gvc = gpu(kc), gpu(vc)
    qo = torch.full(q.shape, 7.0, dtype=BF, device="cuda")
    ko = torch.full(k.shape, 7.0, dtype=BF, device="cuda") if with_k else None
    out = w4.kv_append(gq, gk, gv, gpu(cs, torch.float32), gpu(sn, torch.float32), gkc, gvc, ints(lens), gpu(table, torch.int32),
                       ints(offsets) if use_offsets else None, Q_out=qo, K_out=ko)
    assert out[0] is qo and out[1] is ko
    want_q, want_k, want_kc, want_vc = np.full_like(q, 7), np.full_like(k, 7), kc.copy(), vc.copy()
    SO.append(q, k, v, cs, sn, want_kc, want_vc, lens, table, offsets, want_q, want_k)
    assert np.array_equal(host(qo), want_q, equal_nan=True)
    if with_k:
        assert np.array_equal(host(ko), want_k, equal_nan=True)
    assert np.array_equal(host(gkc), want_kc, equal_nan=True) and np.array_equal(host(gvc), want_vc, equal_nan=True)


@pytest.mark.parametrize("n_q,n_kv,head,page", [(16, 8, 128, 16), (4, 1, 64, 256), (5, 5, 64, 32), (7, 1, 128, 64), (24, 2, 128, 128)])
@pytest.mark.parametrize("new,before", [([1], [0]), ([37, 1, 0, 64, 5], [0, 90, 3, 16, 255]), ([0, 0, 200, 0], [5, 0, 1, 0]), ([3] * 70, [11] * 70), ([1, 0] * 2500, [3, 7] * 2500)])
def test_append(n_q, n_kv, head, page, new, before):
    say("append", n_q, n_kv, head, page, new[:5])
    _run_append(_append_case(np.random.default_rng(len(new) + head), new, before, n_q, n_kv, head, page))


def test_append_one_token_each():
    rng = np.random.default_rng(6)
    before = [0, 1, 15, 16, 17, 31, 2000, 5, 255, 256]
    case = _append_case(rng, [1] * 10, before, 16, 8, 128, 16, spare=0)
    _run_append(case, use_offsets=False, with_k=False)
    _run_append(case, use_offsets=True)


def test_append_leaves_out_what_has_no_place():
    """Positions before 0 and past the angles: no row is written; pages outside the cache or past the table: no slot is."""
    rng = np.random.default_rng(7)
    case = list(_append_case(rng, [4, 6, 2, 5], [10, 14, 30, 0], 4, 2, 64, 16, positions=31))
    case[4] = [14, 20, 32, 2]                                    # the last sequence's first three tokens lie before 0
    table = case[5]
    table[0] = -1
    table[1] = [2 ** 31 - 1, table[1][1]]
    _run_append(tuple(case))
    case = list(_append_case(rng, [4, 40], [10, 0], 4, 2, 64, 16))
    case[5] = case[5][:, :2].copy()                              # the second sequence's third page is past the table
    case[5][0] = len(case[8])
    _run_append(tuple(case))


def test_append_offsets_out_of_range_stay_in_bounds():
    """Descending and outlying offsets: nothing outside the arrays is touched, and tokens of proper sequences come out right."""
    rng = np.random.default_rng(17)
    case = _append_case(rng, [4, 6], [0, 0], 4, 2, 64, 16, spare=0)
    qkv, q, k, v, lens, table, cs, sn, kc, vc, _ = case
    g, qo = gpu(qkv), torch.full(q.shape, 7.0, dtype=BF, device="cuda")
    w4.kv_append(g[:, :4], g[:, 4:6], g[:, 6:], gpu(cs, torch.float32), gpu(sn, torch.float32), gpu(kc), gpu(vc), ints([4, 6]),
                 gpu(table, torch.int32), ints([-5, 4, 2 ** 31 - 1]), Q_out=qo)
    want = np.full_like(q, 7)
    want[:4] = SO.rotate(q[:4], cs[:4], sn[:4])
    want[4:] = SO.rotate(q[4:], cs[:6], sn[:6])
    assert np.array_equal(host(qo), want)
    qo.fill_(7)
    w4.kv_append(g[:, :4], g[:, 4:6], g[:, 6:], gpu(cs, torch.float32), gpu(sn, torch.float32), gpu(kc), gpu(vc), ints([4, 6]),
                 gpu(table, torch.int32), ints([9, 3, -1]), Q_out=qo)
    torch.cuda.synchronize()
    w4.kv_append(g[:, :4], g[:, 4:6], g[:, 6:], gpu(cs, torch.float32), gpu(sn, torch.float32), gpu(kc), gpu(vc), ints([-2 ** 31, 2 ** 31 - 1]),
                 gpu(table, torch.int32), ints([0, 4, 10]), Q_out=qo)
    torch.cuda.synchronize()


def test_append_in_place():
    rng = np.random.default_rng(9)
    q, k, v = normal(rng, 5, 4, 128), normal(rng, 5, 2, 128), normal(rng, 5, 2, 128)
    cs, sn = w4.rope_table(5, 128)
    kc = torch.zeros(1, 2, 16, 128, dtype=BF, device="cuda")
    gq, gk = gpu(q), gpu(k)
    w4.kv_append(gq, gk, gpu(v), cs, sn, kc, kc.clone(), ints([5]), ints([[0]]), ints([0, 5]), Q_out=gq, K_out=gk)
    c, s = cs.cpu().numpy(), sn.cpu().numpy()
    assert np.array_equal(host(gq), SO.rotate(q, c, s)) and np.array_equal(host(gk), SO.rotate(k, c, s))
    assert same_bits(kc[0, :, :5], gk.transpose(0, 1))


def test_append_past_32_bit_offsets():
    """Slots past 2^32 bytes of the cache, tokens past 2^31 elements of the input."""
    rng = np.random.default_rng(10)
    page, n_kv, head = 16, 8, 128
    pages = (5 << 30) // (n_kv * page * head * 2)
    kc = torch.empty(pages, n_kv, page, head, dtype=BF, device="cuda")
    vc = torch.empty_like(kc)
    kc[-3:], vc[-3:] = 3, 3
    base = torch.empty(130 << 24, dtype=BF, device="cuda")
    far = lambda n, at: base.as_strided((130, n, head), (1 << 24, head, 1), at * head)  # noqa: E731
    q, k, v = normal(rng, 130, 8, head), normal(rng, 130, 8, head), normal(rng, 130, 8, head)
    gq, gk, gv = far(8, 0), far(8, 8), far(8, 16)
    gq.copy_(gpu(q)), gk.copy_(gpu(k)), gv.copy_(gpu(v))
    cs, sn = w4.rope_table(200, head)
    table = ints([[i for i in range(10)], [pages - 1 - i for i in range(10)]])
    qo, ko = w4.kv_append(gq, gk, gv, cs, sn, kc, vc, ints([100, 30]), table, ints([0, 100, 130]), K_out=torch.empty_like(gpu(k)))
    c, s = cs.cpu().numpy(), sn.cpu().numpy()
    pos = np.r_[0:100, 0:30]
    want = SO.rotate(k, c[pos], s[pos])
    assert np.array_equal(host(qo), SO.rotate(q, c[pos], s[pos])) and np.array_equal(host(ko), want)
    for p in range(30):
        assert np.array_equal(host(kc[pages - 1 - p // 16, :, p % 16]), want[100 + p])
        assert np.array_equal(host(vc[pages - 1 - p // 16, :, p % 16]), v[100 + p])
    assert (kc[-3] == 3).all() and (kc[-2, :, 14:] == 3).all()


# ---------------------------------------------------------------- attention

class Bounds:
    """Collects one run's elements and holds them to the bounds of this file's head."""

    def __init__(self, head):
        self.head, self.square, self.limit, self.extra, self.n = head, 0.0, 0.0, 0.0, 0

    def add(self, got, q, k, v, scale, visible=None):
        """got, q [m][head] against keys k, v [n][head], fp64; visible [m][n] or None for all."""
        s = scale * (q @ k.T)
        reach = (scale * (q.abs() @ k.abs().T))
        if visible is not None:
            s = s.masked_fill(~visible, -INF)
            reach = reach.masked_fill(~visible, 0)
        p = s.softmax(dim=1)
        o, spread, noise = p @ v, p @ v.abs(), ((p * p) @ (v * v)).sqrt()
        n = len(k)
        e = (reach.amax(dim=1, keepdim=True) * (self.head + 8) * 2.0 ** -23 + 2.0 ** -20) * 2 + 2 * n * 2.0 ** -23
        off = (got - o).abs()
        bound = (2.0 ** -8 + e) * spread + 2.0 ** -8 * o.abs() + 1e-38
        assert not torch.isnan(got).any(), "NaN came out"
        assert (off <= bound).all(), f"off by {(off / bound).max():.3f} of the bound"
        self.square += float((off ** 2).sum())
        self.limit += float(((2.0 ** -8 * noise) ** 2 + (2.0 ** -8 * o) ** 2).sum())
        self.extra += float(((e * spread) ** 2).sum())
        self.n += off.numel()

    def done(self):
        if self.n >= 256:
            assert math.sqrt(self.square) <= math.sqrt(self.limit) + math.sqrt(self.extra), \
                f"rms {math.sqrt(self.square / self.n):.3g} of {math.sqrt(self.limit / self.n):.3g}"


def check_prompt(got, q, k, v, lengths, scale, heads=None):
    got, q, k, v = (t.double().cpu() for t in (got, q, k, v))
    group, c, at = q.shape[1] // k.shape[1], Bounds(q.shape[2]), 0
    for n in lengths:
        if n:
            seen = torch.ones(n, n, dtype=torch.bool).tril()
            for h in range(q.shape[1]) if heads is None else heads:
                c.add(got[at:at + n, h], q[at:at + n, h], k[at:at + n, h // group], v[at:at + n, h // group], scale, seen)
        at += n
    c.done()


def offsets_of(lengths):
    out = [0]
    for n in lengths:
        out.append(out[-1] + n)
    return out


def fused(gen, T, n_q, n_kv, head, scale=1.0):
    qkv = (torch.randn(T, n_q + 2 * n_kv, head, generator=gen, device="cuda") * scale).to(BF)
    return qkv[:, :n_q], qkv[:, n_q:n_q + n_kv], qkv[:, n_q + n_kv:]


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


LENGTHS = [[1], [37], [2, 1], [64], [65, 63], [128, 0, 129], [0, 0, 5, 0], [300, 17, 1, 255, 256, 257], [1] * 40, [513, 31]]


@pytest.mark.parametrize("head", [64, 128])
@pytest.mark.parametrize("n_q,n_kv", [(1, 1), (4, 2), (5, 5), (7, 1), (16, 2)])
@pytest.mark.parametrize("lengths", LENGTHS)
def test_prompt_attention(head, n_q, n_kv, lengths):
    say("prompt", head, n_q, n_kv, lengths[:6])
    T = sum(lengths)
    q, k, v = fused(generator(T + n_q), T + 5, n_q, n_kv, head)
    k[T:], v[T:] = NAN, NAN                                       # rows behind the last sequence
    o = torch.full((T + 5, n_q, head), 7.0, dtype=BF, device="cuda")
    assert w4.prompt_attention(q, k, v, ints(offsets_of(lengths)), O=o) is o
    assert (o[T:] == 7).all()
    check_prompt(o[:T], q[:T], k[:T], v[:T], lengths, head ** -0.5)
    o2 = w4.prompt_attention(q, k, v, ints(offsets_of(lengths)))
    assert same_bits(o[:T], o2[:T])


@pytest.mark.parametrize("head,n_q,n_kv,lengths", [(128, 2, 1, [4099]), (64, 1, 1, [6001, 3]), (128, 3, 1, [1025, 2047]), (128, 16, 8, [700, 900])])
def test_prompt_attention_long(head, n_q, n_kv, lengths):
    say("prompt long", head, n_q, n_kv, lengths)
    T = sum(lengths)
    q, k, v = fused(generator(T), T, n_q, n_kv, head)
    o = w4.prompt_attention(q, k, v, ints(offsets_of(lengths)))
    check_prompt(o, q, k, v, lengths, head ** -0.5, heads=range(min(n_q, 3)))


@pytest.mark.parametrize("head,n_q,n_kv,lengths", [(128, 16, 8, [8300]), (64, 16, 2, [5000, 3300, 1]), (128, 24, 3, [65, 5000, 0, 900]), (64, 17, 17, [7800])])
def test_prompt_attention_many_rows(head, n_q, n_kv, lengths):
    """Past the row count from which eight waves share key tiles: rows at both ends and between, of some heads."""
    say("prompt many rows", head, n_q, n_kv, lengths)
    T = sum(lengths)
    assert T * n_q >= 512 * 256
    q, k, v = fused(generator(T), T, n_q, n_kv, head)
    o = w4.prompt_attention(q, k, v, ints(offsets_of(lengths)))
    assert same_bits(o, w4.prompt_attention(q, k, v, ints(offsets_of(lengths))))
    go, gq, gk, gv = (t.double().cpu() for t in (o, q, k, v))
    c, at, group = Bounds(head), 0, n_q // n_kv
    for n in lengths:
        for h in (0, n_q // 2, n_q - 1):
            for first in sorted({0, max(0, n // 2 - 77), max(0, n - 130)}):
                rows = min(130, n - first)
                if rows <= 0:
                    continue
                seen = torch.arange(first + rows)[None, :] <= torch.arange(first, first + rows)[:, None]
                c.add(go[at + first:at + first + rows, h], gq[at + first:at + first + rows, h], gk[at:at + first + rows, h // group],
                      gv[at:at + first + rows, h // group], head ** -0.5, seen)
        at += n
    c.done()


@pytest.mark.parametrize("lengths", [[3] * 300, [1] * 5000, [0, 2] * 200 + [700] + [5] * 100, [1 + i % 90 for i in range(257)]])
def test_prompt_attention_many_sequences(lengths):
    say("prompt many sequences", len(lengths))
    T = sum(lengths)
    q, k, v = fused(generator(len(lengths)), T + 3, 4, 2, 64)
    o = torch.full((T + 3, 4, 64), 7.0, dtype=BF, device="cuda")
    w4.prompt_attention(q, k, v, ints(offsets_of(lengths)), O=o)
    assert (o[T:] == 7).all()
    check_prompt(o[:T], q[:T], k[:T], v[:T], lengths, 64 ** -0.5, heads=(0, 3))


def test_packed_rows_before_the_first_sequence():
    """offsets[0] > 0: the rows before it belong to no sequence."""
    q, k, v = fused(generator(31), 200, 4, 2, 128)
    k[:50], v[:50] = NAN, NAN
    o = torch.full((200, 4, 128), 7.0, dtype=BF, device="cuda")
    w4.prompt_attention(q, k, v, ints([50, 120, 190]), O=o)
    assert (o[:50] == 7).all() and (o[190:] == 7).all()
    check_prompt(o[50:190], q[50:190], k[50:190], v[50:190], [70, 70], 128 ** -0.5)
    cs, sn = w4.rope_table(100)
    qo = torch.full((200, 4, 128), 7.0, dtype=BF, device="cuda")
    kc = torch.zeros(8, 2, 64, 128, dtype=BF, device="cuda")
    w4.kv_append(q, k, v, cs, sn, kc, torch.zeros_like(kc), ints([70, 70]), ints([[0, 1], [2, 3]]), ints([50, 120, 190]), Q_out=qo)
    assert (qo[:50] == 7).all() and (qo[190:] == 7).all() and not (qo[50:190] == 7).all(dim=2).any() and not kc[4:].any()


@pytest.mark.parametrize("head", [64, 128])
def test_prompt_attention_scales(head):
    """Sharp and flat softmax; scores in the thousands neither overflow nor lose the maximum."""
    q, k, v = fused(generator(head), 300, 4, 2, head)
    for scale in (1e-6, 0.5, 3.0):
        o = w4.prompt_attention(q, k, v, ints([0, 300]), scale=scale)
        check_prompt(o, q, k, v, [300], float(np.float32(scale)))
    big = (q.float() * 40).to(BF)
    o = w4.prompt_attention(big, k, v, ints([0, 300]), scale=1.0)
    # the scores' own rounding swamps the bound here: only the range is held (p and o are rounded, 2^-8 each)
    assert torch.isfinite(o.float()).all() and o.float().abs().max() <= v.float().abs().max() * (1 + 2.0 ** -6)
    # rising scores: every key block raises the maximum; equal scores: the mean of the values
    ramp = torch.arange(300, device="cuda").float()[:, None, None].expand(300, 2, head) / 64
    ones = torch.ones(300, 4, head, dtype=BF, device="cuda")
    for kk in (ramp.to(BF), (-ramp).to(BF), torch.zeros_like(k)):
        o = w4.prompt_attention(ones, kk.contiguous(), v, ints([0, 300]))
        check_prompt(o, ones, kk, v, [300], head ** -0.5)


@pytest.mark.parametrize("head", [64, 128])
@pytest.mark.parametrize("at", [0, 1, 31, 32, 63, 64, 100, 149])
def test_prompt_attention_unseen_values(head, at):
    """NaN and infinities in a later token's key or value, and in other sequences, reach no earlier token."""
    for seed, what in enumerate((NAN, INF, -INF)):
        q, k, v = fused(generator(seed), 150 + 70, 4, 2, head)
        k0, v0 = k.clone(), v.clone()
        k[at, :, 3], v[at, :, 5], v[at, 1, head - 1] = what, what, what
        o = w4.prompt_attention(q, k, v, ints([0, 150, 220]))
        check_prompt(torch.cat((o[:at], o[150:])), torch.cat((q[:at], q[150:])), torch.cat((k0[:at], k0[150:])), torch.cat((v0[:at], v0[150:])),
                     [at, 70], head ** -0.5)
        if math.isnan(what):
            assert torch.isnan(o[at:150].float()).all()            # a NaN score is every later token's
        k[at], v[at] = k0[at], v0[at]
        v[at, :, 5] = what                                         # a value alone: its own channel of later tokens
        o = w4.prompt_attention(q, k, v, ints([0, 150, 220])).float()
        later = o[at:150, :, 5]
        assert torch.isnan(later).all() if math.isnan(what) else (torch.isnan(later) | (later == what)).all()
        o[at:150, :, 5] = 0
        assert torch.isfinite(o).all()


def test_prompt_attention_far_apart_tokens():
    """Tokens 2^24 elements apart: offsets past 2^32 bytes."""
    n, head = 300, 128
    base = torch.empty(n << 24, dtype=BF, device="cuda")
    far = lambda heads, at: base.as_strided((n, heads, head), (1 << 24, head, 1), at * head)  # noqa: E731
    q, k, v = fused(generator(2), n, 4, 2, head)
    gq, gk, gv = far(4, 0), far(2, 4), far(2, 6)
    gq.copy_(q), gk.copy_(k), gv.copy_(v)
    o = w4.prompt_attention(gq, gk, gv, ints([0, 150, 300]))
    assert same_bits(o, w4.prompt_attention(q, k, v, ints([0, 150, 300])))
    check_prompt(o, q, k, v, [150, 150], head ** -0.5)


def test_prompt_attention_offsets_out_of_range_stay_in_bounds():
    q, k, v = fused(generator(3), 100, 4, 2, 128)
    o = w4.prompt_attention(q, k, v, ints([-7, 60, 2 ** 31 - 1]))
    check_prompt(o, q, k, v, [60, 40], 128 ** -0.5)
    for bad in ([50, 20, -3], [2 ** 31 - 1, 0, 100], [100, 100, 0]):
        w4.prompt_attention(q, k, v, ints(bad))
        torch.cuda.synchronize()


def paged(gen, lens, n_kv, head, page, prefix=0, spare=2, stale=NAN):
    """A cache with the sequences' keys and values, everything else `stale`: (k_cache, v_cache, table, keys, values)."""
    width = max(1, max(-(-n // page) for n in lens), prefix // page)
    shared = prefix // page
    need = [max(0, -(-n // page) - shared) for n in lens]
    pages = shared + sum(need) + spare
    order = torch.randperm(pages, generator=gen, device="cuda").tolist()
    kc = torch.full((pages, n_kv, page, head), stale, dtype=BF, device="cuda")
    vc = kc.clone()
    table = [[(-1, 2 ** 31 - 1, pages)[(b + i) % 3] for i in range(width)] for b in range(len(lens))]
    table[0][:shared] = order[:shared]
    common_k = torch.randn(prefix, n_kv, head, generator=gen, device="cuda").to(BF)
    common_v = torch.randn(prefix, n_kv, head, generator=gen, device="cuda").to(BF)
    at, keys, values = shared, [], []

    def put(page_ids, first, k, v):
        for i in range(0, len(k), page):
            kk, vv = k[i:i + page], v[i:i + page]
            kc[page_ids[(first + i) // page], :, :len(kk)] = kk.transpose(0, 1)
            vc[page_ids[(first + i) // page], :, :len(vv)] = vv.transpose(0, 1)

    put(table[0], 0, common_k, common_v)
    for b, n in enumerate(lens):
        own = max(0, n - prefix)
        table[b][shared:shared + need[b]] = order[at:at + need[b]]
        at += need[b]
        k = torch.randn(own, n_kv, head, generator=gen, device="cuda").to(BF)
        v = torch.randn(own, n_kv, head, generator=gen, device="cuda").to(BF)
        put(table[b], prefix, k, v)
        keys.append(torch.cat((common_k[:n], k)))
        values.append(torch.cat((common_v[:n], v)))
    return kc, vc, ints(table), keys, values


def check_decode(got, q, keys, values, scale):
    got, q = got.double().cpu(), q.double().cpu()
    c = Bounds(q.shape[2])
    for b in range(len(keys)):
        k, v = keys[b].double().cpu(), values[b].double().cpu()
        if len(k) == 0:
            assert not got[b].any()
            continue
        group = q.shape[1] // k.shape[1]
        for j in range(k.shape[1]):
            h = slice(j * group, (j + 1) * group)
            c.add(got[b, h], q[b, h], k[:, j], v[:, j], scale)
    c.done()


DECODE = [([1], 0), ([500], 0), ([0, 1, 15, 16, 17, 0, 33, 300], 0), ([257] * 3, 256), ([300, 256, 800, 257, 512], 256), ([2100, 2049], 2048),
          ([1025 + 7 * i for i in range(20)], 1024), ([5, 300, 0, 256, 100, 700], 256), ([4000, 1, 2], 0), ([513] * 70, 512), ([40] * 65, 0), ([260] * 300 + [0] * 10 + [257], 256)]


@pytest.mark.parametrize("head", [64, 128])
@pytest.mark.parametrize("n_q,n_kv,page", [(1, 1, 16), (4, 2, 256), (16, 8, 32), (7, 1, 64), (5, 5, 128), (24, 1, 16), (32, 2, 64)])
@pytest.mark.parametrize("lens,prefix", DECODE)
def test_decode_attention(head, n_q, n_kv, page, lens, prefix):
    say("decode", head, n_q, n_kv, page, lens[:6], prefix)
    gen = generator(len(lens) + n_q)
    kc, vc, table, keys, values = paged(gen, lens, n_kv, head, page, prefix)
    q = fused(gen, len(lens), n_q, n_kv, head)[0]
    o = w4.decode_attention(q, kc, vc, ints(lens), table, max_len=max(lens), prefix_len=prefix)
    check_decode(o, q, keys, values, head ** -0.5)
    # the same from the table's own bound, and once more
    o2 = w4.decode_attention(q, kc, vc, ints(lens), table, prefix_len=prefix)
    check_decode(o2, q, keys, values, head ** -0.5)
    assert same_bits(o, w4.decode_attention(q, kc, vc, ints(lens), table, max_len=max(lens), prefix_len=prefix))


@pytest.mark.parametrize("lens,prefix,n_q,n_kv", [([20000], 0, 4, 1), ([9000 + i for i in range(3)], 8192, 8, 2), ([4200] * 130, 4096, 2, 1)])
def test_decode_attention_long(lens, prefix, n_q, n_kv):
    gen = generator(77)
    kc, vc, table, keys, values = paged(gen, lens, n_kv, 128, 64, prefix)
    q = fused(gen, len(lens), n_q, n_kv, 128)[0]
    o = w4.decode_attention(q, kc, vc, ints(lens), table, max_len=max(lens), prefix_len=prefix)
    check_decode(o, q, keys, values, 128 ** -0.5)


def test_decode_attention_lengths_past_the_bounds():
    """max_len cuts, negative lengths are empty; lengths past the table are never followed."""
    gen = generator(5)
    kc, vc, table, keys, values = paged(gen, [300, 300, 300], 2, 128, 16)
    q = fused(gen, 3, 4, 2, 128)[0]
    o = w4.decode_attention(q, kc, vc, ints([2 ** 31 - 1, -5, 40]), table, max_len=100)
    cut = [t[:n] for t, n in zip(keys, (100, 0, 40))], [t[:n] for t, n in zip(values, (100, 0, 40))]
    check_decode(o, q, *cut, 128 ** -0.5)
    o = w4.decode_attention(q, kc, vc, ints([300, 300, 300]), table, max_len=0)
    assert not o.any()


@pytest.mark.parametrize("prefix", [0, 64])
def test_decode_attention_leaves_out_bad_pages(prefix):
    gen = generator(6)
    lens = [300, 200, 90]
    kc, vc, table, keys, values = paged(gen, lens, 2, 128, 16, prefix)
    q = fused(gen, 3, 4, 2, 128)[0]
    gone = {(0, 1): -1, (0, 17): 2 ** 31 - 1, (1, 5): kc.shape[0], (2, 4): -2 ** 31, (2, 5): 10 ** 9}
    kept = [torch.ones(n, dtype=torch.bool, device="cuda") for n in lens]
    for (b, i), bad in gone.items():
        table[b, i] = bad
        for row in range(3) if b == 0 and i < prefix // 16 else [b]:
            kept[row][16 * i:16 * i + 16] = False
    o = w4.decode_attention(q, kc, vc, ints(lens), table, max_len=300, prefix_len=prefix)
    check_decode(o, q, [k[m] for k, m in zip(keys, kept)], [v[m] for v, m in zip(values, kept)], 128 ** -0.5)
    table[1] = -1                                                  # no key of its own left
    if not prefix:
        assert not w4.decode_attention(q, kc, vc, ints(lens), table, max_len=300)[1].any()


def test_decode_attention_one_infinite_value():
    """A seen infinity or NaN stays in its channel and its sequence."""
    gen = generator(8)
    kc, vc, table, keys, values = paged(gen, [100, 80, 90], 1, 64, 16, 64)
    q = fused(gen, 3, 2, 1, 64)[0]
    vc[table[1, 4].item(), 0, 3, 9] = INF
    o = w4.decode_attention(q, kc, vc, ints([100, 80, 90]), table, max_len=100, prefix_len=64).float()
    assert (o[1, :, 9] == INF).all() and torch.isfinite(o[[0, 2]]).all() and torch.isfinite(o[1, :, :9]).all()


def test_decode_attention_short_rows_under_a_prefix_with_nan():
    """A row shorter than the prefix sees nothing of the prefix's later tokens, whatever they hold."""
    gen = generator(9)
    lens = [400, 70, 256, 3]
    kc, vc, table, keys, values = paged(gen, lens, 2, 128, 64, 256)
    q = fused(gen, 4, 4, 2, 128)[0]
    vc[table[0, 1].item(), 1, 30, 7] = NAN                          # prefix token 94
    kc[table[0, 3].item(), 0, 0, 0] = NAN                           # prefix token 192
    o = w4.decode_attention(q, kc, vc, ints(lens), table, max_len=400, prefix_len=256)
    check_decode(o[[1, 3]], q[[1, 3]], [keys[1], keys[3]], [values[1], values[3]], 128 ** -0.5)
    assert torch.isnan(o[0, :2].float()).all() and torch.isnan(o[0, 2:, 7].float()).all()


@pytest.mark.parametrize("lens,prefix,first,end", [
    ([33], 0, 32, 33), ([300], 0, 288, 300), ([641], 0, 640, 641), ([600, 33, 900], 0, 32, 33), ([300] * 3, 256, 32, 64),
    ([700] * 40, 512, 256, 384), ([4100] * 65, 4096, 0, 1024), ([4100] * 65, 4096, 3968, 4096)])
def test_decode_attention_keys_of_nan_alone_in_their_chunk(lens, prefix, first, end):
    """NaN keys that a sequence sees make all its outputs NaN, also where a wave, a tile or a chunk has no other key."""
    gen = generator(len(lens))
    kc, vc, table, keys, values = paged(gen, lens, 2, 128, 16, prefix)
    q = fused(gen, len(lens), 8, 2, 128)[0]
    for p in range(first, end):
        kc[int(table[0, p // 16]), :, p % 16] = NAN
    o = w4.decode_attention(q, kc, vc, ints(lens), table, max_len=max(lens), prefix_len=prefix)
    hit = len(lens) if prefix else 1
    assert torch.isnan(o[:hit].float()).all()
    check_decode(o[hit:], q[hit:], keys[hit:], values[hit:], 128 ** -0.5)


@pytest.mark.parametrize("lens,prefix,hidden", [([40], 0, 32), ([1100], 0, 128), ([4100] * 65, 4096, 64), ([4100] * 65, 4096, 1100)])
def test_decode_attention_scores_of_minus_infinity(lens, prefix, hidden):
    """The first `hidden` keys of sequence 0 or the prefix have scores of -infinity: a weight of 0, however few keys are left."""
    gen = generator(len(lens) + 1)
    kc, vc, table, keys, values = paged(gen, lens, 2, 128, 16, prefix)
    q = fused(gen, len(lens), 8, 2, 128)[0].clone()
    q[:, :, 0] = q[:, :, 0].abs() + 1
    for p in range(hidden):
        kc[int(table[0, p // 16]), :, p % 16, 0] = -INF
    o = w4.decode_attention(q, kc, vc, ints(lens), table, max_len=max(lens), prefix_len=prefix)
    check_decode(o, q, [k[hidden:] for k in keys], [v[hidden:] for v in values], 128 ** -0.5)


@pytest.mark.parametrize("head", [64, 128])
@pytest.mark.parametrize("n_q", [4, 512])
@pytest.mark.parametrize("low", [-60, -87, -95])
def test_prompt_attention_scores_of_minus_infinity(head, n_q, low):
    """The first tile's scores are -infinity, the others far below 0: those alone count."""
    q, k, v = (t.clone() for t in fused(generator(head), 300, n_q, 2, head))
    q[:, :, 0] = q[:, :, 0].abs() + 1
    q[:, :, 1], k[:, :, 1] = 8, low * head ** 0.5 / 8
    k[:64, :, 0] = -INF
    o = w4.prompt_attention(q, k, v, ints([0, 300]))
    check_prompt(o[64:], q[64:], k[64:], v[64:], [236], head ** -0.5, heads=[0, 1, n_q - 1])


def test_decode_attention_cache_past_32_bits():
    page, n_kv, head = 64, 8, 128
    pages = (5 << 30) // (n_kv * page * head * 2)
    gen = generator(10)
    kc = torch.empty(pages, n_kv, page, head, dtype=BF, device="cuda")
    vc = torch.empty_like(kc)
    small_k, small_v, small_table, keys, values = paged(gen, [300, 150], n_kv, head, page, 64)
    kc[-len(small_k):], vc[-len(small_v):] = small_k, small_v
    q = fused(gen, 2, 16, n_kv, head)[0]
    shift = pages - len(small_k)
    ok = (small_table >= 0) & (small_table < len(small_k))
    table = torch.where(ok, small_table + shift, small_table)
    o = w4.decode_attention(q, kc, vc, ints([300, 150]), table, max_len=300, prefix_len=64)
    assert same_bits(o, w4.decode_attention(q, small_k, small_v, ints([300, 150]), small_table, max_len=300, prefix_len=64))
    check_decode(o, q, keys, values, head ** -0.5)


# ---------------------------------------------------------------- streams, graphs, workspaces

def test_on_another_stream_and_in_graphs():
    """Captured once, replayed with new inputs, lengths and pages, eager work in between; two graphs share a workspace."""
    gen = generator(11)
    lens_a, lens_b = [300, 200, 40, 130], [150, 290, 300, 0]
    prefix, page = 32, 16
    width = 19
    ca, cb = (paged(gen, lens, 2, 128, page, prefix, spare=60 - sum(max(0, -(-n // page) - 2) for n in lens)) for lens in (lens_a, lens_b))
    kc, vc = ca[0].clone(), ca[1].clone()
    table, lens = ca[2].clone(), ints(lens_a)
    q = fused(gen, 4, 8, 2, 128)[0].contiguous()
    outs, graphs = [], []
    w = normal(np.random.default_rng(1), 256)
    gx, gr, gw = torch.zeros(4, 256, dtype=BF, device="cuda"), torch.zeros(4, 256, dtype=BF, device="cuda"), gpu(w)
    first = w4.decode_attention_launcher(q, kc, vc, lens, table, max_len=300, prefix_len=prefix, O=torch.empty_like(q))
    pq, pk, pv = fused(gen, 200, 8, 2, 128)
    pq, pk, pv, off = pq.contiguous(), pk.contiguous(), pv.contiguous(), ints([0, 120, 200])
    stream = torch.cuda.Stream()
    for i in range(2):
        o, po = torch.empty_like(q), torch.empty_like(pq)
        n8 = [torch.empty(4, 256, dtype=torch.int8, device="cuda"), torch.empty(4, device="cuda"), torch.empty(4, 2, dtype=torch.int32, device="cuda"),
              torch.empty(4, 256, dtype=BF, device="cuda")]
        calls = [w4.decode_attention_launcher(q, kc, vc, lens, table, max_len=300, prefix_len=prefix, O=o, workspace=first.workspace),
                 w4.prompt_attention_launcher(pq, pk, pv, off, O=po), w4.w4a8_rmsnorm_launcher(gx, gw, gr, 1e-6, *n8)]
        with torch.cuda.stream(stream):
            for c in calls:
                c()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for c in calls:
                c()
        outs.append((o, po, n8, calls)), graphs.append(g)
    for step in range(4):
        src, src_lens = ((ca, lens_a), (cb, lens_b))[step % 2]
        kc.copy_(src[0]), vc.copy_(src[1]), lens.copy_(ints(src_lens))
        table.fill_(-1)
        table[:, :min(width, src[2].shape[1])] = src[2][:, :table.shape[1]]
        q.copy_(torch.randn(q.shape, generator=gen, device="cuda")), pq.copy_(torch.randn(pq.shape, generator=gen, device="cuda"))
        off.copy_(ints(([0, 120, 200], [0, 1, 140])[step % 2]))
        gx.copy_(torch.randn(4, 256, generator=gen, device="cuda"))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        want = w4.decode_attention(q, kc, vc, lens, table, max_len=300, prefix_len=prefix)
        check_decode(want, q, src[3], src[4], 128 ** -0.5)
        pwant, n = w4.prompt_attention(pq, pk, pv, off), (200, 140)[step % 2]
        nwant = w4.w4a8_rmsnorm(gx, gw, gr, 1e-6)
        for o, po, n8, _ in outs:
            assert same_bits(o, want) and same_bits(po[:n], pwant[:n])
            assert all(torch.equal(a, b) for a, b in zip(n8, nwant))


def test_two_streams_at_once():
    gen = generator(12)
    kc, vc, table, keys, values = paged(gen, [2000, 1800], 2, 128, 16, 1024)
    q = [fused(gen, 2, 4, 2, 128)[0].contiguous() for _ in range(2)]
    want = [w4.decode_attention(x, kc, vc, ints([2000, 1800]), table, max_len=2000, prefix_len=1024) for x in q]
    lens = ints([2000, 1800])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(w4.decode_attention(q[i], kc, vc, lens, table, max_len=2000, prefix_len=1024))
    torch.cuda.synchronize()
    assert all(same_bits(o, want[i]) for i in range(2) for o in got[i])


def test_workspace_of_the_size_asked_for():
    """Nothing behind the workspace's size is touched; one too small is refused."""
    gen = generator(13)
    for lens, prefix, n_q, n_kv in (([3000, 2900], 1024, 8, 2), ([600] * 9, 512, 7, 1), ([5000], 0, 4, 1)):
        kc, vc, table, keys, values = paged(gen, lens, n_kv, 128, 64, prefix)
        q = fused(gen, len(lens), n_q, n_kv, 128)[0].contiguous()
        size = w4.decode_attention_launcher(q, kc, vc, ints(lens), table, max_len=max(lens), prefix_len=prefix).workspace_size
        if size is None:
            continue
        buf = torch.full((size.value + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
        o = w4.decode_attention(q, kc, vc, ints(lens), table, max_len=max(lens), prefix_len=prefix, workspace=buf[:size.value])
        assert (buf[size.value:] == 0xFF).all()
        check_decode(o, q, keys, values, 128 ** -0.5)


def test_binding_refusals_on_the_gpu():
    q = torch.zeros(4, 4, 128, dtype=BF, device="cuda")
    kv = torch.zeros(4, 2, 128, dtype=BF, device="cuda")
    cache = torch.zeros(3, 2, 16, 128, dtype=BF, device="cuda")
    off, lens, table = ints([0, 4]), ints([4, 4, 4, 4]), ints([[0]] * 4)
    cs, sn = w4.rope_table(16)
    with pytest.raises(ValueError):
        w4.prompt_attention(q, kv, kv[:3], off)
    with pytest.raises(ValueError):
        w4.prompt_attention(q.transpose(0, 1).contiguous().transpose(0, 1), kv, kv, off)      # heads of a token apart
    with pytest.raises(TypeError):
        w4.prompt_attention(q.float(), kv, kv, off)
    with pytest.raises(ValueError):
        w4.prompt_attention(q, kv, kv[:, :1], off)
    with pytest.raises(w4.W4Error):
        w4.prompt_attention(q, kv, kv, off, scale=0.0)
    with pytest.raises(w4.W4Error):
        w4.prompt_attention(q[:, :3], kv, kv, off)
    with pytest.raises(ValueError):
        w4.decode_attention(q, cache, cache[:2], lens, table)
    with pytest.raises(ValueError):
        w4.decode_attention(q, cache, cache, lens, table[:3])
    with pytest.raises(ValueError):
        w4.decode_attention(q, cache, cache, lens, table, max_len=-1)
    with pytest.raises(w4.W4Error):
        w4.decode_attention(q, cache, cache, lens, table, max_len=17)
    with pytest.raises(w4.W4Error):
        w4.decode_attention(q, cache, cache, lens, table, prefix_len=8)
    with pytest.raises(ValueError):
        w4.kv_append(q, kv, kv, cs, sn[:3], cache, cache.clone(), lens, table)
    with pytest.raises(ValueError):
        w4.kv_append(q, kv, kv, cs, sn, cache, cache.clone(), lens, table, offsets=lens)
    with pytest.raises(TypeError):
        w4.kv_append(q, kv, kv, cs, sn, cache, cache.clone(), lens.long(), table)
    x, w = torch.zeros(4, 256, dtype=BF, device="cuda"), torch.ones(256, dtype=BF, device="cuda")
    with pytest.raises(ValueError):
        w4.rmsnorm(x, w, H=x)
    with pytest.raises(ValueError):
        w4.rmsnorm(x, w[:128])
    with pytest.raises(w4.W4Error):
        w4.rmsnorm(x, w, eps=-1.0)


# ---------------------------------------------------------------- a run of them together

def _layer(seed, H, n_q, n_kv):
    gen = generator(seed)
    make = lambda n, k: (torch.randn(n, k, generator=gen, device="cuda") * 0.03).to(BF)  # noqa: E731
    blk = {"norm1": (1 + 0.1 * torch.randn(H, generator=gen, device="cuda")).to(BF), "norm2": (1 + 0.1 * torch.randn(H, generator=gen, device="cuda")).to(BF),
           "q": make(128 * n_q, H), "k": make(128 * n_kv, H), "v": make(128 * n_kv, H), "o": make(H, 128 * n_q),
           "gate": make(2 * H, H), "up": make(2 * H, H), "down": make(H, 2 * H)}
    return gen, blk


def test_prompts_as_the_decoder_block():
    """norm, append, prompt attention and norm again, with the block's projections between them, against w4_block_forward."""
    B, L, H, n_q, n_kv = 3, 77, 512, 4, 2
    gen, blk = _layer(21, H, n_q, n_kv)
    X = torch.randn(B * L, H, generator=gen, device="cuda").to(BF)
    want = w4.block_forward(X, B, L, blk, n_q, n_kv)
    off, lens = ints([i * L for i in range(B + 1)]), ints([L] * B)
    cs, sn = w4.rope_table(L)
    kc = torch.zeros(B * 5, n_kv, 16, 128, dtype=BF, device="cuda")
    vc, table = torch.zeros_like(kc), torch.arange(B * 5, dtype=torch.int32, device="cuda").reshape(B, 5)
    a, _ = w4.rmsnorm(X, blk["norm1"])
    qkv = w4.bf16_linear(a, torch.cat((blk["q"], blk["k"], blk["v"]))).reshape(B * L, n_q + 2 * n_kv, 128)
    q, k, v = qkv[:, :n_q], qkv[:, n_q:n_q + n_kv], qkv[:, n_q + n_kv:]
    q, k = w4.kv_append(q, k, v, cs, sn, kc, vc, lens, table, off, K_out=torch.empty(B * L, n_kv, 128, dtype=BF, device="cuda"))
    o = w4.prompt_attention(q, k, v, off)
    p = w4.bf16_linear(o.reshape(B * L, -1), blk["o"])
    b, h = w4.rmsnorm(p, blk["norm2"], residual=X)
    g, u = w4.bf16_linear(b, blk["gate"]).float(), w4.bf16_linear(b, blk["up"]).float()
    y = (h.float() + w4.bf16_linear((g / (1 + torch.exp(-g)) * u).to(BF), blk["down"]).float()).to(BF)
    rel = float((y.double() - want.double()).norm() / want.double().norm())
    assert rel <= 2.0 ** -7, rel
    # the last token of every sequence through the cache gives the same
    last = torch.arange(B, device="cuda") * L + L - 1
    o2 = w4.decode_attention(q[last], kc, vc, lens, table)
    check_decode(o2, q[last], [k[i * L:(i + 1) * L] for i in range(B)], [v[i * L:(i + 1) * L] for i in range(B)], 128 ** -0.5)


def test_decode_step_over_int4_weights():
    """norm to int8, the W4A8 linear for q, k, v, append, attention under a shared prefix, the W4A16 output linear, the next
    norm: every step against 64 bits on the step's own input."""
    B, H, n_q, n_kv, prefix = 6, 512, 4, 2, 64
    gen, blk = _layer(22, H, n_q, n_kv)
    lens = [64 + n for n in (1, 5, 40, 100, 17, 64)]
    kc, vc, table, keys, values = paged(gen, lens, n_kv, 128, 16, prefix)
    X = torch.randn(B, H, generator=gen, device="cuda").to(BF)
    res = torch.randn(B, H, generator=gen, device="cuda").to(BF)
    qw, sc, qz = w4.awq_quantize_pack(torch.cat((blk["q"], blk["k"], blk["v"])))
    ow, osc, oz = w4.awq_quantize_pack(blk["o"])
    Xq, sx, xsum, h = w4.w4a8_rmsnorm(X, blk["norm1"], res)
    _check_norm(host(X), host(res), host(blk["norm1"]), 1e-6, None, h, (Xq, sx, xsum))
    y = w4.w4a8_gemv(Xq, sx, xsum, qw, sc, qz)
    words = lambda t: t.cpu().numpy().view(np.uint32)  # noqa: E731
    bits = lambda t: t.view(torch.int16).cpu().numpy().view(np.uint16)  # noqa: E731
    What = O.dequantize(words(qw), bits(sc), words(qz), H, False).astype(np.float64)
    want = (Xq.cpu().numpy().astype(np.float64) * sx.cpu().numpy()[:, None]) @ What.T
    assert np.linalg.norm(host(y) - want) <= 2.0e-3 * np.linalg.norm(want)
    qkv = y.reshape(B, n_q + 2 * n_kv, 128)
    cs, sn = w4.rope_table(max(lens))
    q, _ = w4.kv_append(qkv[:, :n_q], qkv[:, n_q:n_q + n_kv], qkv[:, n_q + n_kv:], cs, sn, kc, vc, ints(lens), table)
    c, s, pos = cs.cpu().numpy(), sn.cpu().numpy(), np.array(lens) - 1
    assert np.array_equal(host(q), SO.rotate(host(qkv[:, :n_q]), c[pos], s[pos]))
    turned = SO.rotate(host(qkv[:, n_q:n_q + n_kv]), c[pos], s[pos])
    for b in range(B):
        keys[b][-1], values[b][-1] = gpu(turned[b]), qkv[b, n_q + n_kv:]
    o = w4.decode_attention(q, kc, vc, ints(lens), table, prefix_len=prefix)
    check_decode(o, q, keys, values, 128 ** -0.5)
    p = w4.w4a16_gemv(o.reshape(B, -1), ow, osc, oz)
    y2, h2 = w4.rmsnorm(p, blk["norm2"], residual=h)
    _check_norm(host(p), host(h), host(blk["norm2"]), 1e-6, y2, h2)
