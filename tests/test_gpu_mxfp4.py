"""MXFP4 operators on the GPU against the fp64 oracle: codes, scales and expanded values bit
for bit; products within the bound that oracle.mxfp4_oracle.product_bound derives."""
import json

import numpy as np
import pytest
import torch

import weight_only_int4_amd as w4
import workloads as wl
from oracle import mxfp4_oracle as MX
from oracle import w4a16_oracle as O
from tests.gpu_util import bf16_values, bits16, bits32, gpu_available, say, to_bf16, to_f32, to_i32

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs an MI355X GPU")]


def to_u8(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.uint8)).to("cuda")


# ---------------------------------------------------------------- quantize / dequantize

def _check_quantize(W, s=None):
    v = O.bf16_to_f32(W)
    if s is not None:
        v = v * s[None, :]
    codes, byte = MX.quantize(v)
    got_c, got_b = w4.mxfp4_quantize(to_bf16(W), None if s is None else to_f32(s))
    back = w4.mxfp4_dequantize(got_c, got_b)
    torch.cuda.synchronize()
    assert np.array_equal(got_b.cpu().numpy(), byte)
    assert np.array_equal(bits32(got_c), MX.pack(codes))
    want = MX.dequantize(codes, byte)
    got = bf16_values(bits16(back))
    assert np.array_equal(got, want, equal_nan=True)
    ok = ~np.isnan(want)
    assert np.array_equal(np.signbit(got[ok]), np.signbit(want[ok]))


@pytest.mark.parametrize("N,K", [(1, 32), (3, 64), (1, 2048), (7, 96), (16, 2080), (129, 160), (300, 1056), (5, 17408)])
@pytest.mark.parametrize("scaled", [False, True])
def test_quantize(N, K, scaled):
    say("mx quantize", N, K, scaled)
    rng = np.random.default_rng(N * 31 + K)
    W = wl.normal_bf16(rng, (N, K), 0.7)
    s = np.exp(rng.standard_normal(K)).astype(np.float32) if scaled else None
    _check_quantize(W, s)


def test_quantize_every_bf16_value():
    """All 65,536 bit patterns as a block's maximum and as a small element beside larger ones."""
    say("mx quantize every value")
    every = np.arange(65536, dtype=np.uint16)
    W = np.zeros((65536, 32), np.uint16)
    W[:, 0] = every
    W[:, 1] = np.roll(every, 77)
    W[:, 31] = every ^ 0x8000
    with np.errstate(invalid="ignore"):
        _check_quantize(W)


def test_quantize_ties_and_both_ends_of_the_range():
    say("mx quantize ties")
    base = np.array([7.5, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.125, 0.0, -0.0], np.float32)
    rows = []
    for e in (-135, -128, -126, -125, -124, -20, 0, 60, 123, 125):
        with np.errstate(over="ignore"):
            v = np.concatenate([base, -base, base[:8] * 1.0]) * np.float32(2.0) ** np.float32(e)
        rows.append(O.f32_to_bf16(v.astype(np.float32)))
    _check_quantize(np.stack(rows))


def test_quantize_scaled_overflow_and_underflow():
    """s that sends products to infinity, below fp32's normal range, and to NaN."""
    say("mx quantize scaled extremes")
    W = O.f32_to_bf16(np.full((2, 128), 3.0, np.float32))
    s = np.ones(128, np.float32)
    s[0], s[32], s[64], s[96] = 3e38, 1e-44, np.nan, 0.0
    s[33:64] = 1e-44
    with np.errstate(over="ignore", invalid="ignore"):
        _check_quantize(W, s)


def test_dequantize_every_code_and_scale():
    say("mx dequantize table")
    codes = np.tile(np.arange(32, dtype=np.uint8) % 16, (256, 1))
    byte = np.arange(256, dtype=np.uint8)[:, None]
    got = bf16_values(bits16(w4.mxfp4_dequantize(to_i32(MX.pack(codes)), to_u8(byte))))
    want = MX.dequantize(codes, byte)
    want = np.where(np.abs(want) >= 2.0 ** 128, np.copysign(np.inf, want), want)   # past bf16's range
    assert np.array_equal(got, want, equal_nan=True)


def test_quantize_large_offsets():
    """More than 2^31 elements: the last rows of a 4.3 GB weight."""
    say("mx quantize large")
    N, K = 131104, 16416
    W = torch.zeros((N, K), dtype=torch.bfloat16, device="cuda")
    tail = wl.normal_bf16(np.random.default_rng(3), (4, K), 1.0)
    W[-4:] = to_bf16(tail)
    codes, byte = w4.mxfp4_quantize(W)
    del W
    oc, ob = MX.quantize(O.bf16_to_f32(tail))
    assert np.array_equal(bits32(codes[-4:]), MX.pack(oc)) and np.array_equal(byte[-4:].cpu().numpy(), ob)
    assert int(codes[:-4].abs().max()) == 0
    back = w4.mxfp4_dequantize(codes, byte)
    assert np.array_equal(bf16_values(bits16(back[-4:])), MX.dequantize(oc, ob))


# ---------------------------------------------------------------- products

def _weights(rng, N, K):
    """Random codes (all 16) with scales around 2^-7: packed operands and fp64 values."""
    codes = rng.integers(0, 16, (N, K)).astype(np.uint8)
    byte = rng.integers(112, 130, (N, K // 32)).astype(np.uint8)
    return to_i32(MX.pack(codes)), to_u8(byte), MX.dequantize(codes, byte)


def _operands(M, K, N, act, seed=0):
    rng = np.random.default_rng([M, K, N, act, seed])
    qw, sw, W = _weights(rng, N, K)
    if act == 16:
        Xb = wl.normal_bf16(rng, (M, K), 1.0)
        return (to_bf16(Xb),), bf16_values(Xb), qw, sw, W
    qx, sx, X = _weights(rng, M, K)
    return (qx, sx), X, qw, sw, W


def _product(act, acts, qw, sw, **kw):
    return (w4.mxfp4_a16_gemm if act == 16 else w4.mxfp4_a4_gemm)(*acts, qw, sw, **kw)


def _check_product(M, K, N, act):
    acts, X, qw, sw, W = _operands(M, K, N, act)
    # the output sits inside a larger buffer whose other values must stay as they were
    pad = 64
    buf = torch.full((M * N + 2 * pad,), 7.0, dtype=torch.bfloat16, device="cuda")
    Y = buf[pad:pad + M * N].view(M, N)
    _product(act, acts, qw, sw, Y=Y)
    torch.cuda.synchronize()
    ref, bound = MX.product_bound(X, W)
    err = np.abs(bf16_values(bits16(Y)) - ref)
    assert (err <= bound).all(), (err / bound).max()
    assert (buf[:pad] == 7.0).all() and (buf[pad + M * N:] == 7.0).all()


SMALL = [(1, 32, 1), (1, 2048, 2048), (2, 64, 3), (3, 96, 17), (4, 512, 100), (5, 1056, 33), (7, 128, 16),
         (8, 2048, 257), (9, 160, 65), (13, 4128, 31), (16, 6144, 96), (16, 32, 4097), (1, 17408, 130), (12, 5120, 515)]
MEDIUM = [(17, 32, 5), (31, 224, 64), (32, 2048, 130), (33, 1056, 47), (37, 6144, 200), (48, 480, 129), (49, 96, 1),
          (64, 4096, 64), (64, 17408, 72), (65, 1056, 255), (100, 2080, 97)]
LARGE = [(127, 128, 128), (128, 512, 256), (129, 544, 385), (200, 17408, 130), (255, 1056, 257), (256, 256, 512),
         (257, 32, 300), (333, 1056, 2047), (513, 2016, 511), (1000, 640, 1)]


@pytest.mark.parametrize("act", [16, 4])
@pytest.mark.parametrize("M,K,N", SMALL + MEDIUM + LARGE)
def test_product(M, K, N, act):
    say("mx product", M, K, N, act)
    _check_product(M, K, N, act)


@pytest.mark.parametrize("act", [16, 4])
@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8, 9, 16, 17, 32, 33, 64, 65, 128, 129])
def test_product_every_row_count_rule(M, act):
    """Both sides of every row count at which another kernel form takes over."""
    for K, N in ((352, 70), (2048, 320)):
        say("mx product rows", M, K, N, act)
        _check_product(M, K, N, act)


@pytest.mark.parametrize("act", [16, 4])
@pytest.mark.parametrize("M,K,N", [(2048, 2048, 640), (1, 5120, 17408), (16, 17408, 5120), (512, 5120, 1024)])
def test_product_model_sizes(M, K, N, act):
    """Full-length rows of the hidden-2048 and 27B-shaped linears (all rows against fp64 on the GPU)."""
    say("mx product model size", M, K, N, act)
    gen = torch.Generator(device="cuda").manual_seed(M + K)
    W = (torch.randn(N, K, generator=gen, device="cuda") * 0.02).bfloat16()
    X = torch.randn(M, K, generator=gen, device="cuda").bfloat16()
    qw, sw = w4.mxfp4_quantize(W)
    Wd = w4.mxfp4_dequantize(qw, sw).double()
    acts = (X,) if act == 16 else w4.mxfp4_quantize(X)
    Xd = X.double() if act == 16 else w4.mxfp4_dequantize(*acts).double()
    Y = _product(act, acts, qw, sw).double()
    ref = Xd @ Wd.T
    acc = K * 2.0 ** -23 * (Xd.abs() @ Wd.abs().T)
    bound = acc + 2.0 ** -8 * (ref.abs() + acc) + 2.0 ** -134
    assert bool(((Y - ref).abs() <= bound).all())


# Shapes of the tiled form: ragged in every direction, K that ends inside a stage and inside four
# stages, scale rows that need padding, K split over workgroups, one and several rounds.
TILED = [(520, 2080, 1001), (700, 1568, 1003), (257, 4160, 1000), (40, 17408, 1500), (300, 17440, 255), (513, 2016, 2050),
         (1030, 1024, 1026), (2049, 640, 1030), (130, 8192, 1001), (4100, 512, 513), (48, 5120, 5119), (2047, 2048, 3000),
         # a workgroup takes several tiles in turn: four stages and more, K's last stage whole and not
         (2047, 512, 17401), (2047, 480, 17401), (2047, 2016, 17401), (2048, 2048, 17408),
         # the large tiles with one tile per workgroup, K split and not
         (1564, 17344, 2577), (940, 6784, 13941), (8691, 1920, 2764), (668, 9792, 6229)]


def _gpu_reference(X, W):
    """product_bound on the GPU, for shapes whose fp64 product would take long on the host."""
    ref, mag = X @ W.T, X.abs() @ W.abs().T
    acc = X.shape[1] * 2.0 ** -23 * mag
    return ref, acc + 2.0 ** -8 * (ref.abs() + acc) + 2.0 ** -134


def _random_packed(gen, rows, K):
    qw = torch.randint(-2 ** 31, 2 ** 31 - 1, (rows, K // 8), generator=gen, device="cuda", dtype=torch.int32)
    sw = torch.randint(112, 130, (rows, K // 32), generator=gen, device="cuda", dtype=torch.uint8)
    return qw, sw, w4.mxfp4_dequantize(qw, sw).double()


@pytest.mark.parametrize("act", [16, 4])
@pytest.mark.parametrize("M,K,N", TILED)
def test_product_tiled(M, K, N, act):
    say("mx product tiled", M, K, N, act)
    gen = torch.Generator(device="cuda").manual_seed(M + 3 * K + 7 * N)
    qw, sw, W = _random_packed(gen, N, K)
    if act == 16:
        acts = (torch.randn(M, K, generator=gen, device="cuda").bfloat16(),)
        X = acts[0].double()
    else:
        *acts, X = _random_packed(gen, M, K)
    buf = torch.full((M * N + 128,), 7.0, dtype=torch.bfloat16, device="cuda")
    Y = buf[64:64 + M * N].view(M, N)
    _product(act, acts, qw, sw, Y=Y)
    ref, bound = _gpu_reference(X, W)
    assert bool(((Y.double() - ref).abs() <= bound).all())
    assert bool((buf[:64] == 7.0).all()) and bool((buf[64 + M * N:] == 7.0).all())
    again = _product(act, acts, qw, sw, workspace=torch.full((512 << 20,), 0xFF, dtype=torch.uint8, device="cuda"))
    assert torch.equal(Y, again)


# Shapes of the register form on which a workgroup has one to five tiles of 4, 8 or 16 channels, with the last
# workgroup's moved back; K that ends inside a step; K split over workgroups.
STREAM = [(1, 5120, 17411), (3, 2080, 6151), (4, 1536, 9001), (7, 2048, 6145), (13, 5152, 17399), (16, 4096, 12289),
          (21, 4128, 12289), (32, 17408, 5121), (30, 5120, 17403), (27, 8224, 1025), (37, 6176, 2047), (17, 2048, 2049)]


@pytest.mark.parametrize("act", [16, 4])
@pytest.mark.parametrize("M,K,N", STREAM)
def test_product_stream(M, K, N, act):
    test_product_tiled(M, K, N, act)


@pytest.mark.parametrize("act", [16, 4])
@pytest.mark.parametrize("M,K,N", [(520, 2080, 1001), (257, 4160, 1000), (40, 17408, 1500), (2047, 2048, 3000), (2047, 2016, 17401), (940, 6752, 13941)])
def test_product_tiled_special_values(M, K, N, act):
    """NaN scale bytes and non-finite activations in the tiled form, in the first and the last block
    of K: one channel or one row each, and nothing else."""
    say("mx product tiled special", M, K, N, act)
    gen = torch.Generator(device="cuda").manual_seed(1)
    qw, sw, _ = _random_packed(gen, N, K)
    sw[5, 0] = 255
    sw[N - 1, K // 32 - 1] = 255
    if act == 16:
        acts = (torch.randn(M, K, generator=gen, device="cuda").bfloat16(),)
        acts[0][3, 1] = float("nan")
        acts[0][M - 1, K - 1] = float("inf")
    else:
        *acts, _ = _random_packed(gen, M, K)
        acts[1][3, 0] = 255
        acts[1][M - 1, K // 32 - 1] = 255
    Y = _product(act, acts, qw, sw).float()
    assert bool(Y[:, [5, N - 1]].isnan().all())
    rest = torch.ones(M, N, dtype=torch.bool, device="cuda")
    rest[:, [5, N - 1]] = False
    rest[[3, M - 1]] = False
    assert bool(Y[rest].isfinite().all())
    if act == 4:
        assert bool(Y[[3, M - 1]].isnan().all())
    else:
        assert bool(Y[3].isnan().all())
        last = qw[:, -1] >> 28                              # the last channel's codes: +-inf, or NaN where zero
        want_nan = (last & 7) == 0
        want_nan[[5, N - 1]] = True
        assert bool((Y[M - 1].isnan() == want_nan).all())
        assert bool((~Y[M - 1].isfinite()).all())


@pytest.mark.parametrize("act", [16, 4])
def test_product_many_rows_one_channel(act):
    """More row groups than a grid dimension other than the first may have."""
    M, K, N = 4_300_000, 32, 1
    say("mx product many rows", M, act)
    gen = torch.Generator(device="cuda").manual_seed(2)
    qw, sw, W = _random_packed(gen, N, K)
    if act == 16:
        acts = (torch.randn(M, K, generator=gen, device="cuda").bfloat16(),)
        X = acts[0].double()
    else:
        *acts, X = _random_packed(gen, M, K)
    ref, bound = _gpu_reference(X, W)
    assert bool(((_product(act, acts, qw, sw).double() - ref).abs() <= bound).all())


@pytest.mark.parametrize("act", [16, 4])
@pytest.mark.parametrize("M", [1, 3, 6, 16, 40, 70, 300])
def test_product_nan_blocks_stay_in_their_channel(M, act):
    """A weight block with byte 255 makes one channel NaN, an activation block one row; zeros beside them stay."""
    K, N = 1056, 150
    say("mx product nan", M, act)
    acts, X, qw, sw, W = _operands(M, K, N, act, 1)
    rows = {0, M - 1}
    cols = {2, N - 1}
    for n in cols:
        sw[n, (5 * n) % (K // 32)] = 255
    if act == 4:
        for m in rows:
            acts[1][m, 32] = 255
    else:
        for m in rows:
            acts[0][m, 1040] = float("nan") if m else float("inf")
    Y = _product(act, acts, qw, sw).float().cpu().numpy()
    nan_col = np.zeros((M, N), bool)
    nan_col[:, list(cols)] = True
    assert np.isnan(Y[nan_col]).all()
    for m in range(M):
        if m in rows:
            assert (~np.isfinite(Y[m])).all()
        else:
            assert np.isfinite(Y[m][~nan_col[m]]).all()


def test_product_extreme_scales():
    """Scale bytes at both ends of their range, brought back by the other operand."""
    say("mx product extreme scales")
    rng = np.random.default_rng(9)
    for M in (3, 40, 130):
        for lo, hi in ((0, 254), (1, 252), (250, 4)):
            K, N = 160, 40
            cw, cx = rng.integers(0, 16, (N, K)).astype(np.uint8), rng.integers(0, 16, (M, K)).astype(np.uint8)
            bw = np.full((N, K // 32), lo, np.uint8)
            bx = np.full((M, K // 32), hi, np.uint8)
            W, X = MX.dequantize(cw, bw), MX.dequantize(cx, bx)
            ref, bound = MX.product_bound(X, W)
            Y = w4.mxfp4_a4_gemm(to_i32(MX.pack(cx)), to_u8(bx), to_i32(MX.pack(cw)), to_u8(bw))
            assert (np.abs(bf16_values(bits16(Y)) - ref) <= bound).all(), (M, lo, hi)
        # 16-bit activations: subnormal weights times large activations
        Xb = O.f32_to_bf16((rng.standard_normal((M, 160)) * 2.0 ** 100).astype(np.float32))
        W = MX.dequantize(cw, np.full((40, 5), 1, np.uint8))
        ref, bound = MX.product_bound(bf16_values(Xb), W)
        Y = w4.mxfp4_a16_gemm(to_bf16(Xb), to_i32(MX.pack(cw)), to_u8(np.full((40, 5), 1)))
        assert (np.abs(bf16_values(bits16(Y)) - ref) <= bound).all(), M


@pytest.mark.parametrize("act", [16, 4])
def test_product_empty(act):
    acts, _, qw, sw, _ = _operands(4, 64, 8, act)
    none = tuple(a[:0] for a in acts)
    assert tuple(_product(act, none, qw, sw).shape) == (0, 8)
    assert tuple(_product(act, acts, qw[:0], sw[:0]).shape) == (4, 0)


@pytest.mark.parametrize("act", [16, 4])
@pytest.mark.parametrize("M,K,N", [(1, 17408, 512), (16, 17408, 512), (40, 6144, 256), (200, 17408, 256), (300, 2048, 600)])
def test_product_repeats_bit_for_bit(M, K, N, act):
    """The same bits on every call, on another stream, with a dirty workspace and output."""
    say("mx product repeat", M, K, N, act)
    acts, _, qw, sw, _ = _operands(M, K, N, act)
    first = _product(act, acts, qw, sw).clone()
    ws = torch.full((256 << 20,), 0xFF, dtype=torch.uint8, device="cuda")
    Y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    _product(act, acts, qw, sw, Y=Y, workspace=ws)
    assert torch.equal(Y, first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        Y2 = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
        _product(act, acts, qw, sw, Y=Y2, workspace=ws)
    side.synchronize()
    assert torch.equal(Y2, first)


def test_binding_checks_shapes():
    (X,), _, qw, sw, _ = _operands(4, 64, 8, 16)
    (qx, sx), _, _, _, _ = _operands(4, 64, 8, 4)
    with pytest.raises(ValueError):
        w4.mxfp4_a16_gemm(X[:, :48].contiguous(), qw, sw)       # K not a multiple of 32
    with pytest.raises(ValueError):
        w4.mxfp4_a16_gemm(X[:, :32].contiguous(), qw, sw)       # K of another weight
    with pytest.raises(ValueError):
        w4.mxfp4_a16_gemm(X, qw, sw[:, :1].contiguous())
    with pytest.raises(ValueError):
        w4.mxfp4_a16_gemm(X, qw, sw, Y=torch.empty(4, 9, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        w4.mxfp4_a4_gemm(qx, sx[:3], qw, sw)
    with pytest.raises(ValueError):
        w4.mxfp4_a16_gemm(X.t().contiguous().t(), qw, sw)       # not contiguous
    with pytest.raises(ValueError):
        w4.mxfp4_quantize(X, torch.ones(32, device="cuda"))
    with pytest.raises(ValueError):
        w4.mxfp4_quantize(X, codes=torch.empty(4, 7, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        w4.mxfp4_dequantize(qw, sw[:4])
    with pytest.raises(w4.W4Error, match="ALIGN"):
        w4.mxfp4_quantize(torch.empty(4 * 64 + 8, dtype=torch.bfloat16, device="cuda")[4:4 * 64 + 4].view(4, 64))


# ---------------------------------------------------------------- together

def _mlp(X, gate, up, down, act):
    """silu(X Wg^T) * (X Wu^T) Wd^T with every linear in MXFP4."""
    def linear(x, w):
        return w4.mxfp4_a16_gemm(x, *w) if act == 16 else w4.mxfp4_a4_gemm(*w4.mxfp4_quantize(x), *w)
    h = torch.nn.functional.silu(linear(X, gate).float()) * linear(X, up).float()
    return linear(h.bfloat16(), down)


@pytest.mark.parametrize("act", [16, 4])
@pytest.mark.parametrize("M", [1, 24, 160])
def test_feed_forward_together_and_in_a_graph(M, act):
    """Quantize, expand and both products as a feed-forward uses them: eager against the formula step by
    step, then captured once and replayed with new inputs between eager calls."""
    say("mx feed-forward", M, act)
    H, I = 512, 1056
    rng = np.random.default_rng(M)
    ws = [w4.mxfp4_quantize(to_bf16(wl.normal_bf16(rng, s, 0.04))) for s in ((I, H), (I, H), (H, I))]
    X = to_bf16(wl.normal_bf16(rng, (M, H), 1.0))

    def value(t):
        return bf16_values(bits16(t))

    def check(x, w, y):
        xa = value(x) if act == 16 else value(w4.mxfp4_dequantize(*w4.mxfp4_quantize(x)))
        ref, bound = MX.product_bound(xa, value(w4.mxfp4_dequantize(*w)))
        assert (np.abs(value(y) - ref) <= bound).all()

    lin = (lambda x, w: w4.mxfp4_a16_gemm(x, *w)) if act == 16 else (
        lambda x, w: w4.mxfp4_a4_gemm(*w4.mxfp4_quantize(x), *w))
    g, u = lin(X, ws[0]), lin(X, ws[1])
    check(X, ws[0], g)
    check(X, ws[1], u)
    h = (torch.nn.functional.silu(g.float()) * u.float()).bfloat16()
    d = lin(h, ws[2])
    check(h, ws[2], d)
    assert torch.equal(_mlp(X, *ws, act), d)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _mlp(X, *ws, act)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _mlp(X, *ws, act)
    for i in range(4):
        X.copy_(to_bf16(wl.normal_bf16(rng, (M, H), 1.0)))
        want = _mlp(X, *ws, act)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i


def test_two_graphs_and_shared_workspace():
    """Launchers captured into two graphs that use one workspace, replayed in turn on one stream."""
    M, K, N = 8, 17408, 512
    say("mx two graphs")
    items = []
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    for act in (16, 4):
        acts, _, qw, sw, _ = _operands(M, K, N, act)
        Y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
        make = w4.mxfp4_a16_gemm_launcher if act == 16 else w4.mxfp4_a4_gemm_launcher
        launch = make(*acts, qw, sw, Y, workspace=ws)
        launch()
        torch.cuda.synchronize()
        want = Y.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            launch()
        items.append((graph, Y, want, launch))
    for _ in range(3):
        for graph, Y, want, _l in items:
            Y.zero_()
            graph.replay()
        torch.cuda.synchronize()
        for graph, Y, want, _l in items:
            assert torch.equal(Y, want)


def test_convert_mxfp4_checkpoint(tmp_path):
    """The converter's MXFP4 output: bit-exact codes and scales, other tensors copied."""
    from safetensors import safe_open
    from weight_only_int4_amd import convert as C
    say("mx convert")
    src, dst = tmp_path / "src", tmp_path / "dst"
    blocks, vocab, hidden = 1, 256, 256
    wl.write_checkpoint(str(src), blocks=blocks, shards=2, vocab=vocab, hidden=hidden)
    assert C.main([str(src), str(dst), "--format", "mxfp4", "--ignore", r".*q_proj\.weight"]) == 0
    out = {}
    for p in sorted(dst.glob("*.safetensors")):
        with safe_open(str(p), framework="pt") as f:
            assert json.loads(f.metadata()["mxfp4"])["block_size"] == 32
            for k in f.keys():
                out[k] = f.get_tensor(k)
    cfg = json.loads((dst / "mxfp4_config.json").read_text())
    assert not (dst / "w4a16_config.json").exists()
    for i, (name, shape) in enumerate(wl.checkpoint_tensor_list(blocks, vocab, hidden)):
        W = wl.checkpoint_tensor(i, name, shape)
        if C.is_converted(name, shape, [r".*q_proj\.weight"], block=32):
            assert name in cfg["converted"] and name not in out
            qn, sn = C.converted_names(name)
            codes, byte = MX.quantize(O.bf16_to_f32(W))
            assert np.array_equal(out[qn].numpy().view(np.uint32), MX.pack(codes)), name
            assert np.array_equal(out[sn].numpy(), byte), name
        else:
            assert np.array_equal(out[name].view(torch.int16).numpy().view(np.uint16), W), name


@pytest.mark.parametrize("act", [16, 4])
def test_two_streams_at_once(act):
    """Calls on two streams with workspaces of their own do not disturb each other."""
    say("mx product two streams", act)
    gen = torch.Generator(device="cuda").manual_seed(5)
    cases = []
    for M, K, N in ((37, 6176, 2047), (300, 17440, 255)):
        qw, sw, _ = _random_packed(gen, N, K)
        acts = (torch.randn(M, K, generator=gen, device="cuda").bfloat16(),) if act == 16 else _random_packed(gen, M, K)[:2]
        want = _product(act, acts, qw, sw)
        Y = torch.empty_like(want)
        make = w4.mxfp4_a16_gemm_launcher if act == 16 else w4.mxfp4_a4_gemm_launcher
        cases.append((make(*acts, qw, sw, Y), Y, want, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for launch, _, _, stream in cases:
            with torch.cuda.stream(stream):
                launch()
    torch.cuda.synchronize()
    for _, Y, want, _ in cases:
        assert torch.equal(Y, want)
