"""MXFP4 without a GPU: the oracle against hand-worked blocks and a scalar restatement, the
entry points' refusals, and the converter's selection."""
import ctypes
import math

import numpy as np
import pytest
import torch

import weight_only_int4_amd as w4
from oracle import mxfp4_oracle as MX
from weight_only_int4_amd import convert as C

P = ctypes.c_void_p
A = P(0x10000)        # a 16-byte aligned fake device address (never dereferenced)
MIS = P(0x10004)


# ---------------------------------------------------------------- oracle pins

def test_magnitudes_round_to_themselves():
    assert np.array_equal(MX.round_e2m1(MX.MAGNITUDES), np.arange(8))
    assert np.array_equal(MX.round_e2m1(-MX.MAGNITUDES), np.arange(8))


def test_ties_go_to_the_even_code_and_large_values_saturate():
    ties = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.5, 7.99]
    assert MX.round_e2m1(ties).tolist() == [0, 2, 2, 4, 4, 6, 6, 7, 7]
    assert MX.round_e2m1(np.nextafter(ties[:7], 9)).tolist() == [1, 2, 3, 4, 5, 6, 7]
    assert MX.round_e2m1(np.nextafter(ties[:7], 0)).tolist() == [0, 1, 2, 3, 4, 5, 6]


def test_worked_block():
    v = np.zeros((1, 32), np.float32)
    v[0, :6] = [10.0, -3.0, 0.5, -0.49, 1.0, 15.9]
    codes, byte = MX.quantize(v)
    assert byte[0, 0] == 128                       # floor(log2 15.9) - 2 = 1: scale 2
    # 5 -> 4 (tie), -1.5, 0.25 -> 0 (tie), -0.245 -> -0, 0.5, 7.95 -> 6
    assert codes[0, :6].tolist() == [6, 11, 0, 8, 1, 7]
    assert MX.dequantize(codes, byte)[0, :6].tolist() == [8.0, -3.0, 0.0, -0.0, 1.0, 12.0]


def test_scalar_restatement():
    """Element by element in plain Python, over scales up to both ends of bf16's range."""
    rng = np.random.default_rng(5)
    v = (rng.standard_normal((60, 64)) * 2.0 ** rng.integers(-140, 126, (60, 1))).astype(np.float32)
    codes, byte = MX.quantize(v)
    for r in range(60):
        for b in range(2):
            block = [float(x) for x in v[r, 32 * b:32 * b + 32]]
            top = max(abs(x) for x in block)
            e = -127 if top < 2.0 ** -126 else max(math.floor(math.log2(top)) - 2, -127)
            assert byte[r, b] == e + 127
            for i, x in enumerate(block):
                c = int(codes[r, 32 * b + i])
                assert (c >> 3) == (math.copysign(1.0, x) < 0)
                mags = [m * 2.0 ** e for m in MX.MAGNITUDES]
                d = [abs(abs(x) - m) for m in mags]
                if abs(x) >= mags[7]:
                    assert c & 7 == 7
                else:
                    best = [j for j in range(8) if d[j] == min(d)]
                    assert c & 7 == (best[0] if len(best) == 1 or best[0] % 2 == 0 else best[1])


def test_special_blocks():
    v = np.zeros((4, 32), np.float32)
    v[0, 3], v[1, 4], v[2, 5] = np.inf, np.nan, -0.0
    v[3, :2] = [2.0 ** -127, 2.0 ** -129]          # a subnormal maximum
    codes, byte = MX.quantize(v)
    assert byte[:, 0].tolist() == [255, 255, 0, 0]
    assert not codes[:2].any() and codes[2, 5] == 8
    assert codes[3, :3].tolist() == [2, 0, 0]      # 1 and 0.25 times 2^-127
    assert np.isnan(MX.dequantize(codes, byte)[0]).all()


def test_pack_round_trip():
    codes = np.random.default_rng(1).integers(0, 16, (3, 64)).astype(np.uint8)
    words = MX.pack(codes)
    assert words[0, 0] == sum(int(codes[0, j]) << (4 * j) for j in range(8))
    assert np.array_equal(MX.unpack(words), codes)


def test_powers_of_two_move_only_the_scale():
    v = np.random.default_rng(2).standard_normal((5, 96)).astype(np.float32)
    c0, b0 = MX.quantize(v)
    c1, b1 = MX.quantize(v * np.float32(2.0 ** 20))
    assert np.array_equal(c0, c1) and np.array_equal(b0 + 20, b1)
    # values on the grid come back unchanged
    w = MX.dequantize(c0, b0)
    c2, b2 = MX.quantize(w.astype(np.float32))
    assert np.array_equal(MX.dequantize(c2, b2), w)


# ---------------------------------------------------------------- refusals of the C entry points

@pytest.fixture(scope="module")
def lib():
    return w4.load_library()


def test_quantize_refusals(lib):
    f = lib.mxfp4_quantize
    for K in (0, -32, 31, 48):
        assert f(A, 4, K, None, A, A, None) == -2
    assert f(A, -1, 64, None, A, A, None) == -2
    assert f(A, 2 ** 31 - 1, 32, None, A, A, None) == -2
    assert f(None, 4, 64, None, A, A, None) == -1
    assert f(A, 4, 64, None, None, A, None) == -1
    assert f(A, 4, 64, None, A, None, None) == -1
    for i in (0, 3, 4, 5):
        args = [A, 4, 64, A, A, A, None]
        args[i] = MIS
        assert f(*args) == -3
    assert f(None, 0, 64, None, None, None, None) == 0


def test_dequantize_refusals(lib):
    f = lib.mxfp4_dequantize
    assert f(A, A, 4, 40, A, None) == -2
    assert f(A, A, -4, 64, A, None) == -2
    assert f(A, A, 2 ** 31 - 1, 32, A, None) == -2
    for i in (0, 1, 4):
        args = [A, A, 4, 64, A, None]
        args[i] = None
        assert f(*args) == -1
        args[i] = MIS
        assert f(*args) == -3
    assert f(None, None, 0, 64, None, None) == 0


def _gemm_calls(lib):
    a16 = lambda M, K, N, x=A, xs=A, w=A, s=A, y=A, ws=None, sz=None: lib.mxfp4_a16_gemm(x, M, K, N, w, s, y, ws, sz, None)
    a4 = lambda M, K, N, x=A, xs=A, w=A, s=A, y=A, ws=None, sz=None: lib.mxfp4_a4_gemm(x, xs, M, K, N, w, s, y, ws, sz, None)
    return (("a16", a16), ("a4", a4))


def test_gemm_refusals(lib):
    sz = ctypes.c_size_t(0)
    for name, f in _gemm_calls(lib):
        for M, K, N in ((-1, 64, 8), (1, 0, 8), (1, 33, 8), (1, 64, -1), (1, (1 << 21) + 32, 8), (2 ** 31 - 1, 32, 1),
                        (1, 32, 2 ** 31 - 1), (1 << 30, 32, 1 << 30), (1 << 20, 2080, 1 << 29)):
            assert f(M, K, N) == -2, (name, M, K, N)
            assert f(M, K, N, sz=ctypes.byref(sz)) == -2
        for kw in (dict(x=None), dict(w=None), dict(s=None), dict(y=None)) + ((dict(xs=None),) if name == "a4" else ()):
            assert f(1, 64, 8, **kw) == -1, (name, kw)
        for kw in (dict(x=MIS), dict(w=MIS), dict(s=MIS), dict(y=MIS)) + ((dict(xs=MIS),) if name == "a4" else ()):
            assert f(1, 64, 8, **kw) == -3, (name, kw)
        assert f(0, 64, 8, x=None, y=None) == 0
        assert f(8, 64, 0, w=None, y=None) == 0


def test_gemm_workspace(lib):
    """The size query enqueues nothing; a shape that needs a workspace refuses to run without one."""
    for name, f in _gemm_calls(lib):
        for M, K, N in ((1, 2048, 2048), (16, 17408, 512), (64, 17408, 64), (200, 17408, 128), (2048, 2048, 6144)):
            sz = ctypes.c_size_t(12345)
            assert f(M, K, N, x=None, xs=None, w=None, s=None, y=None, sz=ctypes.byref(sz)) == 0
            need = sz.value
            if need:
                assert f(M, K, N) == -5, (name, M, K, N)
                short = ctypes.c_size_t(need - 1)
                assert f(M, K, N, ws=A, sz=ctypes.byref(short)) == -5
                exact = ctypes.c_size_t(need)
                assert f(M, K, N, ws=MIS, sz=ctypes.byref(exact)) == -3


def test_binding_refuses_host_tensors_and_wrong_types():
    W = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU tensor"):
        w4.mxfp4_quantize(W)
    with pytest.raises(TypeError):
        w4.mxfp4_quantize(W.float())
    with pytest.raises(TypeError):
        w4.mxfp4_dequantize(W, W)
    with pytest.raises(TypeError):
        w4.mxfp4_a16_gemm(W.half(), W, W)
    with pytest.raises(TypeError):
        w4.mxfp4_a4_gemm(W, W, W, W)


# ---------------------------------------------------------------- converter

def test_converter_selects_by_block():
    name = "model.layers.0.mlp.down_proj.weight"
    assert C.is_converted(name, (64, 96), block=w4.MX_BLOCK)
    assert not C.is_converted(name, (64, 96))                  # int4 groups are 128 channels
    assert not C.is_converted(name, (64, 100), block=w4.MX_BLOCK)
    assert not C.is_converted("model.embed_tokens.weight", (64, 96), block=w4.MX_BLOCK)


def test_converter_refuses_unknown_format(tmp_path):
    with pytest.raises(ValueError, match="format"):
        C.convert_checkpoint(str(tmp_path), str(tmp_path / "out"), fmt="int3")


# ---------------------------------------------------------------- the binding's own checks

class _OnGpu(torch.Tensor):
    """A tensor without storage that the binding takes for one on a GPU."""
    is_cuda = True


def _huge(shape, dtype):
    return torch.empty(shape, dtype=dtype, device="meta").as_subclass(_OnGpu)


def _no_call(*args):
    raise AssertionError("the library was called")


@pytest.fixture
def no_library_call(monkeypatch):
    """Any call that gets past the checks fails the test."""
    monkeypatch.setattr(w4, "_mx_call", _no_call)
    monkeypatch.setattr(w4, "_workspace", _no_call)


_BIG = 2 ** 32            # as a C int: 0, so 2^32 + 32 would pass for 32


def test_binding_refuses_sizes_past_an_int(no_library_call):
    """Sizes are int in the C interface; a larger one would lose its upper bits on the way."""
    i32, u8, bf16 = torch.int32, torch.uint8, torch.bfloat16
    for rows, K in ((1, _BIG + 32), (1, 2 ** 31), (_BIG + 4, 32), (2 ** 31, 32)):
        with pytest.raises(ValueError, match="2147483647"):
            w4.mxfp4_quantize(_huge((rows, K), bf16))
        with pytest.raises(ValueError, match="2147483647"):
            w4.mxfp4_dequantize(_huge((rows, K // 8), i32), _huge((rows, K // 32), u8))
        small_q, small_s = _huge((4, K // 8), i32), _huge((4, K // 32), u8)
        with pytest.raises(ValueError, match="2147483647"):
            w4.mxfp4_a16_gemm(_huge((rows, K), bf16), small_q, small_s)
        with pytest.raises(ValueError, match="2147483647"):
            w4.mxfp4_a4_gemm(_huge((rows, K // 8), i32), _huge((rows, K // 32), u8), small_q, small_s)
    for N in (_BIG + 4, 2 ** 31):
        q, s = _huge((N, 8), i32), _huge((N, 2), u8)
        with pytest.raises(ValueError, match="2147483647"):
            w4.mxfp4_a16_gemm(_huge((1, 64), bf16), q, s)
        with pytest.raises(ValueError, match="2147483647"):
            w4.mxfp4_a4_gemm(_huge((1, 8), i32), _huge((1, 2), u8), q, s)


def test_binding_without_the_direct_device_calls(monkeypatch):
    """A torch without the two direct calls takes the public ones."""
    import importlib.util
    monkeypatch.delattr(torch._C, "_cuda_getDevice", raising=False)
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    spec = importlib.util.spec_from_file_location("binding_without_direct_calls", w4.__file__)
    binding = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(binding)

    class Stream:
        def __init__(self, index):
            self.cuda_stream = 100 + index

    entered = []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            entered.append(self.index)

        def __exit__(self, *exc):
            return False

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda index: Stream(index))
    monkeypatch.setattr(torch.cuda, "device", Device)
    seen = []
    for index in (1, 2):
        binding._mx_call(lambda *args: seen.append(args) or 0, (7, 8), index)
    assert seen == [(7, 8, 101), (7, 8, 102)]
    assert entered == [2]                      # only for a device that is not the current one


def test_few_rows_need_no_padded_scales(lib):
    """Up to 24 rows a product does not copy a whole weight's scales first, whatever K (a size query of 0)."""
    for name, f in _gemm_calls(lib):
        for M in (1, 3, 4, 8, 16, 17, 24):
            for K, N in ((2880, 201088), (2080, 151936), (5152, 400000), (480, 1000003), (17440, 65536)):
                sz = ctypes.c_size_t(1)
                assert f(M, K, N, x=None, xs=None, w=None, s=None, y=None, sz=ctypes.byref(sz)) == 0
                assert sz.value == 0, (name, M, K, N)
