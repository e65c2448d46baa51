"""The norms over the whole range of bf16: the mean of squares of finite rows neither overflows nor underflows.

Tolerances as in test_gpu_serve.py: the sum of squares is the same one of values scaled by a power of two."""
import numpy as np
import pytest

import weight_only_int4_amd as w4
from oracle import serve_oracle as SO
from tests import test_gpu_serve as S
from tests.gpu_util import gpu_available, say

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs an MI355X GPU")]


def rows_of(rng, H, exponents):
    """A row of magnitude 2^e for each e, within (-2, 2) 2^e and none of them all zero."""
    x = np.clip(rng.standard_normal((len(exponents), H)), -1.9, 1.9)
    x[:, 0] = 1.5
    return SO.bf16(x * 2.0 ** np.asarray(exponents, np.float64)[:, None])


def check_int8(x, w, eps, int8):
    """_check_norm's bound for codes, sums and scales, and half a step of the smallest numbers for a subnormal scale."""
    with np.errstate(all="ignore"):
        codes, sx, xsum = SO.rmsnorm_int8(x, w, eps)
    assert np.array_equal(int8[0].cpu().numpy(), codes) and np.array_equal(int8[2].cpu().numpy(), xsum)
    got, rel = int8[1].cpu().numpy().astype(np.float64), ((x.shape[1] / 64 + 16) / 2 + 6) * 2.0 ** -24
    assert np.isfinite(sx).all() and np.isfinite(got).all()
    off = np.abs(got - sx)
    assert (off <= rel * sx + 2.0 ** -150).all(), np.flatnonzero(off > rel * sx + 2.0 ** -150)


@pytest.mark.parametrize("H", [128, 1024, 8320, 65536])
@pytest.mark.parametrize("eps", [0.0, 1e-40, 1e-31, 1e-20, 1e-6, 1e20])
def test_rows_of_every_magnitude(H, eps):
    say("norm range", H, eps)
    rng = np.random.default_rng(H)
    x = rows_of(rng, H, range(-133, 127, 1 if H < 8192 else 7))
    w = SO.bf16(1 + 0.2 * rng.standard_normal(H))
    eps32 = float(np.float32(eps))
    y, _ = w4.rmsnorm(S.gpu(x), S.gpu(w), None, eps)
    S._check_norm(x, None, w, eps32, y)
    *int8, _ = w4.w4a8_rmsnorm(S.gpu(x), S.gpu(w), None, eps)
    check_int8(x, w, eps32, int8)


@pytest.mark.parametrize("H", [128, 2048, 17408])
def test_a_few_large_values_in_a_row(H):
    """One value from the top of the range, or a sum with a residual that reaches it, beside ordinary ones; the rows
    next to it are as without it."""
    rng = np.random.default_rng(H + 1)
    x, res = S.normal(rng, 9, H), S.normal(rng, 9, H)
    x[1, 3], x[3, H - 1], x[5, 64], x[7, 7] = 2.0 ** 64, -2.0 ** 127, SO.bf16([3.3e38])[0], 2.0 ** 126
    res[7, 7] = 2.0 ** 126
    w = SO.bf16(1 + 0.2 * rng.standard_normal(H))
    for r in (None, res):
        y, h = w4.rmsnorm(S.gpu(x), S.gpu(w), None if r is None else S.gpu(r), 1e-6)
        S._check_norm(x, r, w, 1e-6, y, h)
        small = SO.bf16(w / 4)                                     # (3.3e38 times 1.6 would be no finite product)
        *int8, h = w4.w4a8_rmsnorm(S.gpu(x), S.gpu(small), None if r is None else S.gpu(r), 1e-6)
        S._check_norm(x, r, small, 1e-6, None, h, int8)
        even = [0, 2, 4, 6, 8]
        y2, _ = w4.rmsnorm(S.gpu(x[even]), S.gpu(w), None if r is None else S.gpu(r[even]), 1e-6)
        assert S.same_bits(y[even], y2)


def test_scales_of_ties_and_quotients():
    """The rows of test_w4a8_rmsnorm_ties_and_scales and test_w4a8_rmsnorm_quotients_next_to_halves, scales included."""
    rng = np.random.default_rng(8)
    x = np.zeros((254, 256), np.float32)
    for i, e in enumerate(range(-126, 128)):
        x[i] = SO.bf16(rng.integers(-254, 255, 256) / 2.0 * 2.0 ** min(e, 120) * 2.0 ** -7)
        x[i, 0] = 127 * 2.0 ** min(e, 120) * 2.0 ** -7
    x = SO.bf16(x)
    w = np.ones(256, np.float32)
    *int8, _ = w4.w4a8_rmsnorm(S.gpu(x), S.gpu(w), None, 0.0)
    S._check_norm(x, None, w, 0.0, None, None, int8)
    y, _ = w4.rmsnorm(S.gpu(x), S.gpu(w), None, 0.0)
    S._check_norm(x, None, w, 0.0, y)
    rng = np.random.default_rng(81)
    x = S.normal(rng, 2048, 1024) * np.float32(2.0) ** rng.integers(-90, 90, (2048, 1)).astype(np.float32)
    x, w = SO.bf16(x), SO.bf16(1 + 0.5 * rng.standard_normal(1024))
    *int8, _ = w4.w4a8_rmsnorm(S.gpu(x), S.gpu(w), None, 0.0)
    S._check_norm(x, None, w, 0.0, None, None, int8)


def test_weights_far_from_one():
    """Scales whose factors alone would leave fp32: steps near the top with large rows, small weights, tiny rows."""
    rng = np.random.default_rng(4)
    for ex, ew in ((100, 27), (126, -100), (126, -130), (-60, 120), (-130, 127), (-130, 0), (0, 126), (60, 60), (-70, -30)):
        x, w = rows_of(rng, 2048, [ex] * 3), rows_of(rng, 2048, [ew])[0] / 2
        w = SO.bf16(w)
        *int8, _ = w4.w4a8_rmsnorm(S.gpu(x), S.gpu(w), None, 0.0)
        check_int8(x, w, 0.0, int8)
