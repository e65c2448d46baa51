"""Cases of the MXFP4 operators (4-bit microscaling floats): quantisation, its inverse and
the two products, each in a plain torch form and through the library.

Format: blocks of 32 input channels share one power-of-two scale 2^(byte - 127); an
element is a sign and one of the magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6 (code 0..7, sign in
bit 3), eight codes per 32-bit word, the first in the lowest bits.

`own` False: `run` computes the plain form in 32 bits and rounds once.  `own` True: `run`
calls the library.
"""
from __future__ import annotations

import torch

own = False

BLOCK = 32
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DEVICE = "cuda"


def listed():
    """The measured cases."""
    return [
        # a decode batch's activations, quantised for the 4-bit product: latency
        dict(name="quantize 16x2048", op="quantize", rows=16, k=2048, s=False),
        # a prefill chunk's activations into the feed-forward's down projection, odd row count
        dict(name="quantize 2047x6144", op="quantize", rows=2047, k=6144, s=False),
        # a large weight with its AWQ input scales, as the converter sees it
        dict(name="quantize 17408x5120 scaled", op="quantize", rows=17408, k=5120, s=True),
        # one small projection of a stored checkpoint, expanded to bf16
        dict(name="dequantize 1024x2048", op="dequantize", rows=1024, k=2048),
        # a large projection of a stored checkpoint, expanded to bf16
        dict(name="dequantize 5120x17408", op="dequantize", rows=5120, k=17408),
        # decode of one sequence through the output projection: latency
        dict(name="a16 1x2048x2048", op="a16", m=1, k=2048, n=2048),
        # a full decode batch through a large feed-forward projection
        dict(name="a16 16x5120x17408", op="a16", m=16, k=5120, n=17408),
        # a ragged batch between decode and prefill, down projection
        dict(name="a16 37x6144x2048", op="a16", m=37, k=6144, n=2048),
        # prefill of 2048 tokens through the gate projection
        dict(name="a16 2048x2048x6144", op="a16", m=2048, k=2048, n=6144),
        # a decode batch with 4-bit activations through the gate projection: latency
        dict(name="a4 8x2048x6144", op="a4", m=8, k=2048, n=6144),
        # odd sizes everywhere: the last blocks of a tile in all three directions
        dict(name="a4 333x1056x2047", op="a4", m=333, k=1056, n=2047),
        # prefill of 2048 tokens through a large feed-forward projection
        dict(name="a4 2048x5120x17408", op="a4", m=2048, k=5120, n=17408),
    ]


def _log_int(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def _draw_k(rng):
    # half of the input sizes are whole 128s as most models have them, half any multiple of a block
    if rng.random() < 0.5:
        return 128 * _log_int(rng, 1, 136)
    return BLOCK * _log_int(rng, 1, 544)


def draw(rng):
    """One more case of the same ranges."""
    op = rng.choice(("quantize", "dequantize", "a16", "a4"))
    while True:
        k = _draw_k(rng)
        if op in ("quantize", "dequantize"):
            rows = _log_int(rng, 1, 17408)
            if 2048 <= rows * k <= 17408 * 5120:
                case = dict(op=op, rows=rows, k=k)
                if op == "quantize":
                    case["s"] = rng.random() < 0.5
                return case
            continue
        m = _log_int(rng, 1, 4096) if rng.random() < 0.5 else _log_int(rng, 1, 64)
        n = _log_int(rng, 1, 17408)
        top = 2048 * 2048 * 6144 if op == "a16" else 2048 * 5120 * 17408
        if n * k >= 65536 and n * k <= 5120 * 17408 and m * n * k <= top:
            return dict(op=op, m=m, k=k, n=n)


# ------------------------------------------------------------------ plain form

def _power_of_two(e):
    """2^e in fp32 for whole e in [-126, 127], from its bit pattern: exact."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _times_power(x, e):
    """x * 2^e for |e| <= 127, in two factors that fp32 holds without loss."""
    half = torch.div(e, 2, rounding_mode="floor")
    return x * _power_of_two(half) * _power_of_two(e - half)


def _plain_quantize(v):
    """fp32 [R][K] -> (codes uint8 [R][K], scale bytes uint8 [R][K/32])."""
    r, k = v.shape
    b = v.reshape(r, k // BLOCK, BLOCK)
    amax = b.abs().amax(dim=2)
    exponent = torch.frexp(amax).exponent - 1                      # floor(log2 amax)
    exponent = torch.where(amax > 0, (exponent - 2).clamp(-127, 127), -127)
    y = _times_power(b.abs(), -exponent[..., None])
    code = torch.zeros(b.shape, dtype=torch.uint8, device=v.device)
    # borders between neighbours; a value on a border goes to the even code
    for border, up_on_tie in ((0.25, 0), (0.75, 1), (1.25, 0), (1.75, 1), (2.5, 0), (3.5, 1), (5.0, 0)):
        code += (y >= border) if up_on_tie else (y > border)
    code |= torch.signbit(b).to(torch.uint8) << 3
    return code.reshape(r, k), (exponent + 127).to(torch.uint8)


def _plain_pack(code):
    """codes uint8 [R][K] -> int32 words [R][K/8], the first code in the lowest bits."""
    r, k = code.shape
    c = code.reshape(r, k // 8, 4, 2)
    return (c[..., 0] | (c[..., 1] << 4)).contiguous().view(torch.int32).reshape(r, k // 8)


def _plain_dequantize(words, scales):
    """int32 words [R][K/8], uint8 scales [R][K/32] -> fp32 [R][K]."""
    r = words.shape[0]
    pairs = words.contiguous().view(torch.uint8).reshape(r, -1)
    codes = torch.stack((pairs & 15, pairs >> 4), dim=2).reshape(r, -1)
    table = torch.tensor(MAGNITUDES + tuple(-x for x in MAGNITUDES), dtype=torch.float32, device=words.device)
    values = table[codes.int()].reshape(r, -1, BLOCK)
    return _times_power(values, scales.int()[..., None] - 127).reshape(r, -1)


def _plain_run(state):
    case = state["case"]
    if case["op"] == "quantize":
        v = state["x"].float()
        if state["s"] is not None:
            v = v * state["s"]
        codes, scales = _plain_quantize(v)
        return _plain_dequantize(_plain_pack(codes), scales).to(torch.bfloat16)
    if case["op"] == "dequantize":
        return _plain_dequantize(state["qw"], state["sw"]).to(torch.bfloat16)
    weight = _plain_dequantize(state["qw"], state["sw"])
    x = state["x"].float() if case["op"] == "a16" else _plain_dequantize(state["qx"], state["sx"])
    return (x @ weight.t()).to(torch.bfloat16)


# ------------------------------------------------------------------ inputs

def _weight(gen, rows, k):
    return (torch.randn(rows, k, generator=gen, device=DEVICE) * 0.02).to(torch.bfloat16)


def _activations(gen, rows, k):
    # one channel in a hundred is twenty times as large, as trained models have them
    x = torch.randn(rows, k, generator=gen, device=DEVICE)
    outlier = torch.rand(k, generator=gen, device=DEVICE) < 0.01
    return (x * (1.0 + 19.0 * outlier.float())).to(torch.bfloat16)


def _packed(v):
    codes, scales = _plain_quantize(v.float())
    return _plain_pack(codes), scales.contiguous()


def _inputs(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    out = {}
    if case["op"] == "quantize":
        if case["s"]:
            out["x"] = _weight(gen, case["rows"], case["k"])
            out["s"] = torch.exp(0.5 * torch.randn(case["k"], generator=gen, device=DEVICE))
        else:
            out["x"], out["s"] = _activations(gen, case["rows"], case["k"]), None
    elif case["op"] == "dequantize":
        out["qw"], out["sw"] = _packed(_weight(gen, case["rows"], case["k"]))
    else:
        out["qw"], out["sw"] = _packed(_weight(gen, case["n"], case["k"]))
        x = _activations(gen, case["m"], case["k"])
        if case["op"] == "a16":
            out["x"] = x
        else:
            out["qx"], out["sx"] = _packed(x)
    return out


def prepare(case, seed):
    """Inputs on the GPU; with `own`, the output buffers and launchers that a serving loop keeps."""
    state = _inputs(case, seed)
    state["case"] = case
    if not own:
        return state
    import weight_only_int4_amd as w4

    state["w4"] = w4
    op = case["op"]
    if op in ("quantize", "dequantize"):
        rows, k = case["rows"], case["k"]
        state["values"] = torch.empty(rows, k, dtype=torch.bfloat16, device=DEVICE)
        if op == "quantize":
            state["codes"] = torch.empty(rows, k // 8, dtype=torch.int32, device=DEVICE)
            state["scales"] = torch.empty(rows, k // BLOCK, dtype=torch.uint8, device=DEVICE)
        return state
    state["y"] = torch.empty(case["m"], case["n"], dtype=torch.bfloat16, device=DEVICE)
    if op == "a16":
        state["launch"] = w4.mxfp4_a16_gemm_launcher(state["x"], state["qw"], state["sw"], state["y"])
    else:
        state["launch"] = w4.mxfp4_a4_gemm_launcher(state["qx"], state["sx"], state["qw"], state["sw"], state["y"])
    return state


def run(state):
    """One pass."""
    if not own:
        return _plain_run(state)
    op = state["case"]["op"]
    if op == "quantize":
        w4 = state["w4"]
        w4.mxfp4_quantize(state["x"], state["s"], codes=state["codes"], scales=state["scales"])
        return w4.mxfp4_dequantize(state["codes"], state["scales"], W=state["values"])
    if op == "dequantize":
        return state["w4"].mxfp4_dequantize(state["qw"], state["sw"], W=state["values"])
    state["launch"]()
    return state["y"]


def work(case):
    """Bytes and operations that one pass cannot do without."""
    packed = 0.5 + 1.0 / BLOCK                                    # bytes of a stored element
    if case["op"] == "quantize":
        n = case["rows"] * case["k"]
        # values in, codes and scales out, and the values they stand for
        return {"bytes": int(n * (2 + packed + 2)) + (4 * case["k"] if case["s"] else 0), "flops": 3 * n}
    if case["op"] == "dequantize":
        n = case["rows"] * case["k"]
        return {"bytes": int(n * (packed + 2)), "flops": n}
    m, k, n = case["m"], case["k"], case["n"]
    x = 2 * m * k if case["op"] == "a16" else int(m * k * packed)
    return {"bytes": int(n * k * packed) + x + 2 * m * n, "flops": 2 * m * n * k}


# ------------------------------------------------------------------ the definition in 64 bits

def _power_of_two_64(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_values(words, scales):
    """sign * (m/2 or (1 + m/2) 2^(e-1)) * 2^(byte-127), from the code's own bit fields."""
    r = words.shape[0]
    shifts = torch.arange(0, 32, 4, device=words.device)
    code = (words.long()[:, :, None] >> shifts) & 15
    sign = 1.0 - 2.0 * (code >> 3).double()
    e, m = (code >> 1) & 3, (code & 1).double()
    mag = torch.where(e == 0, 0.5 * m, (1.0 + 0.5 * m) * _power_of_two_64(e - 1))
    scale = _power_of_two_64(scales.long() - 127)
    return ((sign * mag).reshape(r, -1, BLOCK) * scale[..., None]).reshape(r, -1)


def _exact_rounded(v):
    """The values that 64-bit v [R][K] becomes: multiples of the step around each magnitude."""
    r, k = v.shape
    b = v.reshape(r, k // BLOCK, BLOCK)
    top = b.abs().amax(dim=2, keepdim=True)
    # floor(log2 top): the exponent field of its 64-bit form
    shared = ((top.view(torch.int64) >> 52) & 2047) - 1023
    scale = _power_of_two_64((shared - 2).clamp(-127, 127))
    y = b / scale
    step = torch.where(y.abs() < 2, 0.5, torch.where(y.abs() < 4, 1.0, 2.0)).double()
    q = (torch.round(y / step) * step).clamp(-6.0, 6.0)            # round: halves to even
    return (q * scale).reshape(r, k)


def exact(case, seed):
    """What `run` returns, from the definition in 64 bits."""
    inp = _inputs(case, seed)
    if case["op"] == "quantize":
        v = inp["x"].double()
        if inp["s"] is not None:
            v = (v * inp["s"].double()).float().double()           # the definition's 32-bit product
        return _exact_rounded(v)
    weight = _exact_values(inp["qw"], inp["sw"])
    if case["op"] == "dequantize":
        return weight
    x = inp["x"].double() if case["op"] == "a16" else _exact_values(inp["qx"], inp["sx"])
    return x @ weight.t()
