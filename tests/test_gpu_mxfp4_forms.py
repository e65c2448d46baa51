"""MXFP4 on the GPU, kernel by kernel: every form of the products at the shapes of tests.mx_forms, products whose
workspace is in use captured and replayed, NaN patterns, and the rounding of arbitrary fp32 products."""
import numpy as np
import pytest
import torch

import weight_only_int4_amd as w4
import workloads as wl
from oracle import mxfp4_oracle as MX
from oracle import w4a16_oracle as O
from tests import mx_forms
from tests import test_gpu_mxfp4 as base
from tests.gpu_util import bits32, gpu_available, say, to_bf16, to_f32

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs an MI355X GPU")]


def _operands(M, K, N, act):
    gen = torch.Generator(device="cuda").manual_seed(M + 3 * K + 7 * N)
    qw, sw, W = base._random_packed(gen, N, K)
    if act == 16:
        acts = (torch.randn(M, K, generator=gen, device="cuda").bfloat16(),)
        return acts, acts[0].double(), qw, sw, W
    *acts, X = base._random_packed(gen, M, K)
    return tuple(acts), X, qw, sw, W


def _tile_rms(square):
    """Root mean square over tiles of 16 x 16 outputs (what is left of them at the edges)."""
    mean = torch.nn.functional.avg_pool2d(square[None, None], 16, ceil_mode=True)
    return mean[0, 0].sqrt()


def _check_tiles(Y, X, W):
    """Root mean square error of every 16 x 16 outputs.

    The operands are independent and of mean zero, so a partial sum of an output has at most the variance
    S^2 = sum (x w)^2 of the whole.  Each of at most K additions is off by at most 2^-23 of its partial sum
    (truncation), all in one direction at worst: K 2^-23 S, taken twice because a tile's mean square scatters.
    Rounding to bf16 adds half a step, 2^-8 of the value at most.  Where K is long this is far below
    product_bound: one block of 17,408 channels left out is an error of 0.043 S, the bound 0.0081 S."""
    K = X.shape[1]
    ref = X @ W.T
    spread = (X * X) @ (W * W).T
    acc = 2.0 * K * 2.0 ** -23 * _tile_rms(spread)
    bound = acc + 2.0 ** -8 * (_tile_rms(ref * ref) + acc) + 2.0 ** -134
    err = _tile_rms((Y.double() - ref) ** 2)
    assert bool((err <= bound).all()), float((err / bound).max())


@pytest.mark.parametrize("act,M,K,N,plan", mx_forms.STREAM + mx_forms.TILE)
def test_product_form(act, M, K, N, plan):
    say("mx form", act, M, K, N, plan)
    acts, X, qw, sw, W = _operands(M, K, N, act)
    buf = torch.full((M * N + 128,), 7.0, dtype=torch.bfloat16, device="cuda")
    Y = buf[64:64 + M * N].view(M, N)
    base._product(act, acts, qw, sw, Y=Y)
    ref, bound = base._gpu_reference(X, W)
    assert bool(((Y.double() - ref).abs() <= bound).all())
    _check_tiles(Y, X, W)
    assert bool((buf[:64] == 7.0).all()) and bool((buf[64 + M * N:] == 7.0).all())
    again = base._product(act, acts, qw, sw, workspace=torch.full((512 << 20,), 0xFF, dtype=torch.uint8, device="cuda"))
    assert torch.equal(Y, again)


@pytest.mark.parametrize("act", [16, 4])
@pytest.mark.parametrize("M,K,N", [(1, 17408, 515), (16, 17408, 700), (40, 17408, 1500), (200, 17408, 1030), (1300, 17408, 2050)])
def test_product_long_rows_by_tile(M, K, N, act):
    """The longest rows of the 27B-shaped linears, where product_bound is wide."""
    say("mx long rows", M, K, N, act)
    acts, X, qw, sw, W = _operands(M, K, N, act)
    _check_tiles(base._product(act, acts, qw, sw), X, W)


SPECIAL = [(16, 65, 5120, 17407), (16, 65, 8192, 9001), (16, 96, 2080, 17401), (16, 37, 6176, 2047), (16, 575, 3232, 539),
           (16, 19, 4160, 2138), (4, 129, 17408, 6144), (4, 603, 8928, 377), (4, 505, 7104, 562), (4, 1626, 992, 1247),
           (4, 46, 7648, 1042), (4, 32, 2880, 20000)]


@pytest.mark.parametrize("act,M,K,N", SPECIAL)
def test_product_form_special_values(act, M, K, N):
    base.test_product_tiled_special_values(M, K, N, act)


@pytest.mark.parametrize("M,K,N", [(3, 2080, 70), (37, 6176, 2047), (65, 8192, 9001), (200, 17408, 130), (1069, 1696, 1955)])
def test_every_kind_of_nan_stays_a_nan(M, K, N):
    """Quiet and signalling bf16 NaNs of both signs, smallest and largest payload, with K split over workgroups and not."""
    say("mx nan patterns", M, K, N)
    (X,), _, qw, sw, _ = _operands(M, K, N, 16)
    rows = {0: 0x7F81, 1: 0xFF81, 2: 0x7FFF, M - 1: 0xFFFF}
    for i, (m, bits) in enumerate(rows.items()):
        X.view(torch.int16)[m, (i * 977) % K] = np.uint16(bits).astype(np.int16).item()
    Y = w4.mxfp4_a16_gemm(X, qw, sw)
    nan = Y.isnan().all(dim=1)
    want = torch.zeros(M, dtype=torch.bool, device="cuda")
    want[list(rows)] = True
    assert torch.equal(nan, want)
    assert bool(Y[~want].isfinite().all())


# ---------------------------------------------------------------- workspaces in graphs

WITH_WORKSPACE = [(16, 37, 6176, 2047), (16, 65, 8192, 9001), (16, 575, 3232, 539), (4, 40, 17408, 1500), (4, 513, 2016, 2050),
                  (4, 46, 7648, 1042)]


def _launcher(act, acts, qw, sw, Y, **kw):
    return (w4.mxfp4_a16_gemm_launcher if act == 16 else w4.mxfp4_a4_gemm_launcher)(*acts, qw, sw, Y, **kw)


def test_graphs_that_share_a_workspace_in_use():
    """Launchers that pad scale rows or split K, captured into a graph each with one workspace between them, replayed in
    turn with new activations, other work and eager calls between the replays."""
    say("mx graphs with workspace")
    gen = torch.Generator(device="cuda").manual_seed(11)
    ws = torch.full((64 << 20,), 0xFF, dtype=torch.uint8, device="cuda")
    items = []
    for act, M, K, N in WITH_WORKSPACE:
        acts, _, qw, sw, _ = _operands(M, K, N, act)
        Y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
        launch = _launcher(act, acts, qw, sw, Y, workspace=ws)
        assert launch.workspace_size is not None and launch.workspace_size.value == ws.numel()
        launch()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            launch()
        items.append((act, acts, qw, sw, Y, graph, launch))
    for i in range(4):
        wants = []
        for act, acts, qw, sw, _, _, _ in items:
            if act == 16:
                acts[0].copy_(torch.randn(acts[0].shape, generator=gen, device="cuda").bfloat16())
            else:
                acts[0].copy_(torch.randint(-2 ** 31, 2 ** 31 - 1, acts[0].shape, generator=gen, device="cuda", dtype=torch.int32))
            wants.append(base._product(act, acts, qw, sw))
        ws.fill_(0xFF)
        for *_, Y, graph, _l in items:
            Y.fill_(float("nan"))
            graph.replay()
        torch.cuda.synchronize()
        for (act, acts, *_r), want, item in zip(items, wants, items):
            assert torch.equal(item[4], want), (i, act, want.shape)


@pytest.mark.parametrize("act,M,H,I", [(16, 37, 6176, 2080), (16, 300, 2016, 4128), (4, 300, 2016, 4128), (4, 40, 17408, 1504)])
def test_feed_forward_with_workspaces_in_a_graph(act, M, H, I):
    """As the feed-forward test, at sizes whose products take a workspace from the graph's own memory."""
    say("mx feed-forward with workspaces", act, M, H, I)
    rng = np.random.default_rng(M)
    ws = [w4.mxfp4_quantize(to_bf16(wl.normal_bf16(rng, s, 0.04))) for s in ((I, H), (I, H), (H, I))]
    X = to_bf16(wl.normal_bf16(rng, (M, H), 1.0))
    acts = (X,) if act == 16 else w4.mxfp4_quantize(X)
    probe = _launcher(act, acts, *ws[0], torch.empty(M, I, dtype=torch.bfloat16, device="cuda"))
    assert probe.workspace_size is not None
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        base._mlp(X, *ws, act)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = base._mlp(X, *ws, act)
    for i in range(4):
        X.copy_(to_bf16(wl.normal_bf16(rng, (M, H), 1.0)))
        want = base._mlp(X, *ws, act)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i


# ---------------------------------------------------------------- rounding

def _blocks(top, values):
    """Blocks of 32 fp32 values, `top` first in each, that hold all of `values`."""
    values = np.concatenate([values, np.zeros(-len(values) % 31, np.float32)]).reshape(-1, 31)
    return np.concatenate([np.full((len(values), 1), top, np.float32), values], axis=1).reshape(-1)


def test_quantize_fp32_values_next_to_the_borders():
    """fp32 values v = 1 * s at the seven borders between magnitudes, one and more steps of fp32 to either side, and as
    far off as a format between fp32 and e2m1 might round; at every scale, those of subnormal values among them."""
    say("mx quantize borders")
    borders = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    offsets = np.concatenate([[0.0], *([2.0 ** -j, -2.0 ** -j] for j in range(6, 25)), [3 * 2.0 ** -24, -3 * 2.0 ** -24]])
    near = (borders[:, None] * (1.0 + offsets[None, :])).reshape(-1)
    near = np.concatenate([near, np.nextafter(borders.astype(np.float32), np.float32(9)).astype(np.float64),
                           np.nextafter(borders.astype(np.float32), np.float32(0)).astype(np.float64)])
    near = np.concatenate([near, -near, [6.0, 6.5, 7.0, 7.5, 7.999, -7.999]])
    parts = []
    for e in range(-140, 126):                                  # the block's scale where that is at least 2^-127
        scaled = np.ldexp(near, e)
        parts.append(_blocks(np.float32(np.ldexp(7.0, e)), scaled.astype(np.float32)))
    s = np.concatenate(parts)
    assert np.isfinite(s).all() and s.size % 32 == 0
    for sign in (1.0, -1.0):
        W = O.f32_to_bf16(np.full((1, s.size), sign, np.float32))
        v = (np.float32(sign) * s)[None, :]
        codes, byte = MX.quantize(v)
        got_c, got_b = w4.mxfp4_quantize(to_bf16(W), to_f32(s))
        assert np.array_equal(got_b.cpu().numpy(), byte)
        assert np.array_equal(bits32(got_c), MX.pack(codes))


def test_quantize_every_bf16_value_at_every_scale():
    """At each scale byte 0 to 252 every bf16 value from an eighth of the scale to eight times it, and each larger one as
    the block's maximum."""
    say("mx quantize every value and scale")
    mantissa = np.arange(128, dtype=np.uint32)
    rows = []
    for byte in range(253):
        values = []
        for field in range(max(byte - 3, 0), byte + 2):          # exponent fields below the block maximum's
            values.append(field << 7 | mantissa)
        top = (byte + 2) << 7
        values = np.concatenate(values)
        values = np.concatenate([values, values | 0x8000, top | mantissa, top | mantissa | 0x8000])
        values = np.concatenate([values, np.zeros(-len(values) % 31, np.uint32)]).reshape(-1, 31)
        block = np.concatenate([np.full((len(values), 1), top, np.uint32), values], axis=1).reshape(-1)
        rows.append(np.concatenate([block, np.zeros(2048 - len(block), np.uint32)]))
    W = np.stack(rows).astype(np.uint16)
    codes, byte = MX.quantize(O.bf16_to_f32(W))
    assert (byte[:, 0] == np.arange(253)).all()
    got_c, got_b = w4.mxfp4_quantize(to_bf16(W))
    assert np.array_equal(got_b.cpu().numpy(), byte)
    assert np.array_equal(bits32(got_c), MX.pack(codes))


# ---------------------------------------------------------------- the largest sizes

def _whole_numbers(gen, rows, K):
    """Operands of -1, 0 and 1 (codes 10, 0 and 2), packed with scale 1 and as int8: any sum of up to 2^24
    products is exact in fp32, whatever the order."""
    v = torch.randint(-1, 2, (rows, K), generator=gen, device="cuda", dtype=torch.int8)
    code = torch.tensor([10, 0, 2], dtype=torch.uint8, device="cuda")[(v + 1).int()].view(rows, K // 2, 2)
    packed = (code[..., 0] | code[..., 1] << 4).contiguous().view(torch.int32)
    return packed, torch.full((rows, K // 32), 127, dtype=torch.uint8, device="cuda"), v


def _whole_operands(gen, M, K, N, act):
    qw, sw, W = _whole_numbers(gen, N, K)
    qx, sx, X = _whole_numbers(gen, M, K)
    return ((X.bfloat16(),) if act == 16 else (qx, sx)), X, qw, sw, W


def _exactly(Y, X, W):
    return torch.equal(Y, (X.double() @ W.double().T).bfloat16())


@pytest.mark.parametrize("act", [16, 4])
@pytest.mark.parametrize("M,N", [(1, 70), (7, 70), (20, 45), (40, 130), (300, 260)])
def test_product_longest_rows(M, N, act):
    """K = 2^21, the most that the products take."""
    K = 1 << 21
    say("mx longest rows", M, N, act)
    acts, X, qw, sw, W = _whole_operands(torch.Generator(device="cuda").manual_seed(M), M, K, N, act)
    assert _exactly(base._product(act, acts, qw, sw), X, W)


@pytest.mark.parametrize("act", [16, 4])
@pytest.mark.parametrize("M,K,N", [(8, 32, 300_000_001), (65, 1024, 5_000_001), (50_000, 64, 50_001), (70, 96, 40_000_001)])
def test_product_offsets_past_32_bits(M, K, N, act):
    """Weights of more than 2^31 bytes and outputs of more than 2^31 elements: the first and last rows and channels."""
    say("mx offsets past 32 bits", M, K, N, act)
    gen = torch.Generator(device="cuda").manual_seed(N)
    acts, X, qw, sw, W = _whole_operands(gen, M, K, N, act)
    Y = base._product(act, acts, qw, sw)
    for m in (slice(0, 300), slice(max(0, M - 300), M)):
        for n in (slice(0, 700), slice(N // 2, N // 2 + 700), slice(N - 700, N)):
            assert _exactly(Y[m, n], X[m], W[n])
