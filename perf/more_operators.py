"""Cases of the operators between a decoder's quantized linears when it serves: the norm with
the residual's addition (bf16 or int8 out), rotary embedding with the append to a paged cache,
causal attention over packed prompts, and attention of single tokens over the paged cache with a
prefix that the batch shares; each in a plain torch form and through the library.

Caches are [pages][kv heads][page size][head size] bf16.  Sequence b's tokens lie in the packed
arrays at offsets[b] .. offsets[b + 1], and its cache holds lens[b] tokens, token p in slot
p % page_size of page table[b][p // page_size].

`own` False: `run` computes the plain form in 32 bits and rounds once.  `own` True: `run`
calls the library.
"""
from __future__ import annotations

import random

import torch

own = False

DEVICE = "cuda"
GROUP = 128          # channels of an int8 code sum
EPS = 1e-6
ROPE_BASE = 1e6


def listed():
    """The measured cases."""
    return [
        # decode of one sequence, into the int8 linears: latency
        dict(name="norm8 1x2048", op="norm8", rows=1, hidden=2048),
        # the rows of one calibration or prompt batch, into 16-bit linears
        dict(name="norm 4096x2048", op="norm", rows=4096, hidden=2048),
        # a long prompt of the wide model, int8, odd row count
        dict(name="norm8 8191x5120", op="norm8", rows=8191, hidden=5120),
        # a decode batch of 16 sequences: one token each, behind contexts of different lengths
        dict(name="append 16x1 page 16", op="append", seqs=16, new=1, before=2000, ragged=1, n_kv=8, group=2, head=128, page=16),
        # a batch of whole prompts of different lengths
        dict(name="append 8x2048 page 64", op="append", seqs=8, new=2048, before=0, ragged=2, n_kv=8, group=4, head=128, page=64),
        # one short prompt: latency
        dict(name="prompt 1x37", op="prompt", seqs=1, longest=37, ragged=0, n_kv=8, group=2, head=128),
        # eight equal sequences, as the block calibration has them
        dict(name="prompt 8x512", op="prompt", seqs=8, longest=512, ragged=0, n_kv=8, group=2, head=128),
        # prompts of different odd lengths, small heads
        dict(name="prompt 12x2047 ragged head 64", op="prompt", seqs=12, longest=2047, ragged=3, n_kv=8, group=4, head=64),
        # one long prompt
        dict(name="prompt 1x8192", op="prompt", seqs=1, longest=8192, ragged=0, n_kv=8, group=2, head=128),
        # one sequence, short context, nothing shared: latency
        dict(name="decode 1x500", op="decode", seqs=1, prefix=0, longest=500, ragged=0, n_kv=8, group=2, head=128, page=16),
        # 16 answers under one system prompt
        dict(name="decode 16x512 prefix 2048", op="decode", seqs=16, prefix=2048, longest=512, ragged=4, n_kv=8, group=2, head=128, page=16),
        # a full batch over a long shared document, answers of different lengths
        dict(name="decode 64x2000 prefix 8192", op="decode", seqs=64, prefix=8192, longest=2000, ragged=5, n_kv=8, group=4, head=128, page=64),
    ]


def _log_int(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    """One more case of the same ranges."""
    op = rng.choice(("norm", "norm8", "append", "prompt", "prompt", "decode", "decode"))
    while True:
        if op in ("norm", "norm8"):
            case = dict(op=op, rows=_log_int(rng, 1, 8191), hidden=GROUP * _log_int(rng, 2, 136))
            if case["rows"] * case["hidden"] <= 8191 * 5120:
                return case
            continue
        heads = dict(n_kv=rng.choice((1, 2, 4, 5, 8, 16)), group=rng.choice((1, 2, 3, 4, 5, 7, 8, 16)), head=rng.choice((64, 128, 128)))
        if heads["n_kv"] * heads["group"] > 64:
            continue
        ragged = rng.choice((0, rng.randrange(1, 1000), rng.randrange(1, 1000)))
        if op == "append":
            new = 1 if rng.random() < 0.5 else _log_int(rng, 2, 2048)
            case = dict(op=op, seqs=_log_int(rng, 1, 128), new=new, before=rng.choice((0, _log_int(rng, 1, 4096))), ragged=ragged,
                        page=rng.choice((16, 32, 64, 128)), **heads)
            if case["seqs"] * (new + case["before"]) * heads["n_kv"] * heads["head"] > 1 << 27:
                continue
            if work(case)["bytes"] <= 190 << 20:
                return case
            continue
        if op == "prompt":
            case = dict(op=op, seqs=_log_int(rng, 1, 32), longest=_log_int(rng, 1, 8192), ragged=ragged, **heads)
            # the plain form's padded scores
            if case["seqs"] * heads["n_kv"] * heads["group"] * case["longest"] ** 2 > 1 << 30:
                continue
            if work(case)["flops"] <= 4 * 128 * 16 * 8192 * 8193 // 2:
                return case
            continue
        page = rng.choice((16, 32, 64, 128))
        prefix = page * (_log_int(rng, 1, 16384 // page) if rng.random() < 0.7 else 0)
        case = dict(op=op, seqs=_log_int(rng, 1, 256), prefix=prefix, longest=_log_int(rng, 1, 8192), ragged=ragged, page=page, **heads)
        # the plain form gathers every sequence's whole context
        if case["seqs"] * (prefix + case["longest"]) * heads["n_kv"] * heads["head"] > 1 << 30:
            continue
        if work(case)["bytes"] <= 288 << 20:
            return case


# ------------------------------------------------------------------ lengths of a case

def _lengths(seqs, longest, ragged):
    """Lengths of the sequences: all `longest`, or (ragged > 0, which picks them) the first of
    them `longest` and the others anything from one token to that."""
    if not ragged:
        return [longest] * seqs
    rng = random.Random(ragged)
    return [longest] + [rng.randint(1, longest) for _ in range(seqs - 1)]


def _offsets(lengths):
    out = [0]
    for n in lengths:
        out.append(out[-1] + n)
    return out


def _cache_lens(case):
    """(tokens of this call, tokens in the cache after it) per sequence."""
    if case["op"] == "append":
        new = [1] * case["seqs"] if case["new"] == 1 else _lengths(case["seqs"], case["new"], case["ragged"])
        before = _lengths(case["seqs"], case["before"], case["ragged"] + 1) if case["before"] else [0] * case["seqs"]
        return new, [a + b for a, b in zip(new, before)]
    own_lens = _lengths(case["seqs"], case["longest"], case["ragged"])
    return [1] * case["seqs"], [case["prefix"] + n for n in own_lens]


# ------------------------------------------------------------------ inputs

def _activations(gen, rows, k):
    # one channel in a hundred is twenty times as large, as trained models have them
    x = torch.randn(rows, k, generator=gen, device=DEVICE)
    outlier = torch.rand(k, generator=gen, device=DEVICE) < 0.01
    return (x * (1.0 + 19.0 * outlier.float())).to(torch.bfloat16)


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEVICE).to(torch.bfloat16)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEVICE)


def _pages(gen, case, lens):
    """Table [sequences][pages] of a lived-in cache: pages in no order, some of them free."""
    page, shared = case["page"], case.get("prefix", 0) // case["page"]
    width = max(-(-n // page) for n in lens)
    total = shared + sum(-(-n // page) - shared for n in lens) + 8
    order = torch.randperm(total, generator=gen, device=DEVICE).to(torch.int32)
    take, rows = shared, []
    for n in lens:
        count = -(-n // page) - shared
        rows.append(list(range(shared)) + list(range(take, take + count)) + [total - 1] * (width - shared - count))
        take += count
    return order[torch.tensor(rows, device=DEVICE)].contiguous(), total


def _inputs(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    out = {}
    if case["op"] in ("norm", "norm8"):
        out["x"] = _activations(gen, case["rows"], case["hidden"])
        out["residual"] = _activations(gen, case["rows"], case["hidden"])
        out["weight"] = (1.0 + 0.1 * torch.randn(case["hidden"], generator=gen, device=DEVICE)).to(torch.bfloat16)
        return out
    n_kv, n_q, head = case["n_kv"], case["n_kv"] * case["group"], case["head"]
    if case["op"] == "prompt":
        offsets = _offsets(_lengths(case["seqs"], case["longest"], case["ragged"]))
        tokens = offsets[-1]
        out["offsets"] = _ints(offsets)
        out["longest"] = case["longest"]
        out["q"], out["k"], out["v"] = _normal(gen, tokens, n_q, head), _normal(gen, tokens, n_kv, head), _normal(gen, tokens, n_kv, head)
        return out
    new, lens = _cache_lens(case)
    out["table"], total = _pages(gen, case, lens)
    out["lens"] = _ints(lens)
    out["k_cache"] = _normal(gen, total, n_kv, case["page"], head)
    out["v_cache"] = _normal(gen, total, n_kv, case["page"], head)
    if case["op"] == "append":
        offsets = _offsets(new)
        tokens = offsets[-1]
        out["offsets"] = _ints(offsets)
        # queries, keys and values side by side, as one projection writes them
        qkv = _normal(gen, tokens, n_q + 2 * n_kv, head)
        out["q"], out["k"], out["v"] = qkv[:, :n_q], qkv[:, n_q:n_q + n_kv], qkv[:, n_q + n_kv:]
        positions = torch.arange(max(lens), device=DEVICE, dtype=torch.float64)
        frequency = ROPE_BASE ** (-2.0 * torch.arange(head // 2, device=DEVICE, dtype=torch.float64) / head)
        angle = positions[:, None] * frequency
        out["cos"], out["sin"] = angle.cos().float().contiguous(), angle.sin().float().contiguous()
        return out
    out["q"] = _normal(gen, case["seqs"], n_q, head)
    out["longest"] = max(lens)
    out["prefix"] = case["prefix"]
    return out


def prepare(case, seed):
    """Inputs on the GPU; with `own`, the output buffers and launchers that a serving loop keeps."""
    state = _inputs(case, seed)
    state["op"] = case["op"]
    if not own:
        return state
    import weight_only_int4_amd as w4

    op = case["op"]
    if op == "norm":
        x = state["x"]
        state["out"] = (torch.empty_like(x), torch.empty_like(x))
        state["launch"] = w4.rmsnorm_launcher(x, state["weight"], state["residual"], EPS, *state["out"])
    elif op == "norm8":
        x, rows, hidden = state["x"], case["rows"], case["hidden"]
        state["codes"] = torch.empty(rows, hidden, dtype=torch.int8, device=DEVICE)
        state["out"] = (torch.empty(rows, dtype=torch.float32, device=DEVICE),
                        torch.empty(rows, hidden // GROUP, dtype=torch.int32, device=DEVICE), torch.empty_like(x))
        state["launch"] = w4.w4a8_rmsnorm_launcher(x, state["weight"], state["residual"], EPS, state["codes"], *state["out"])
    elif op == "append":
        q_out = torch.empty(state["q"].shape, dtype=torch.bfloat16, device=DEVICE)
        k_out = torch.empty(state["k"].shape, dtype=torch.bfloat16, device=DEVICE)
        state["out"] = (q_out, k_out, state["k_cache"], state["v_cache"])
        state["launch"] = w4.kv_append_launcher(state["q"], state["k"], state["v"], state["cos"], state["sin"], state["k_cache"],
                                                state["v_cache"], state["lens"], state["table"], state["offsets"], q_out, k_out)
    elif op == "prompt":
        state["out"] = torch.empty_like(state["q"])
        state["launch"] = w4.prompt_attention_launcher(state["q"], state["k"], state["v"], state["offsets"], O=state["out"])
    else:
        state["out"] = torch.empty_like(state["q"])
        state["launch"] = w4.decode_attention_launcher(state["q"], state["k_cache"], state["v_cache"], state["lens"], state["table"],
                                                       max_len=state["longest"], prefix_len=state["prefix"], O=state["out"])
    return state


def run(state):
    """One pass."""
    if own:
        state["launch"]()
        if state["op"] == "norm8":
            # the codes are whole numbers that the definition fixes bit for bit, and are returned as such
            return (state["codes"], *state["out"])
        return state["out"]
    return {"norm": _plain_norm, "norm8": _plain_norm8, "append": _plain_append, "prompt": _plain_prompt, "decode": _plain_decode}[state["op"]](state)


# ------------------------------------------------------------------ plain forms

def _plain_sum(state):
    h = (state["x"].float() + state["residual"].float()).to(torch.bfloat16)
    f = h.float()
    return h, f, 1.0 / torch.sqrt((f * f).mean(dim=1, keepdim=True) + EPS)


def _plain_norm(state):
    h, f, r = _plain_sum(state)
    return (f * r * state["weight"].float()).to(torch.bfloat16), h


def _plain_norm8(state):
    h, f, r = _plain_sum(state)
    v = f * state["weight"].float()                                # exact: 8-bit significands
    top = v.abs().amax(dim=1, keepdim=True)
    t = torch.where(top > 0, top / 127.0, 1.0)
    # the 32-bit quotient, correctly rounded by way of 64 bits
    codes = torch.round((v.double() / t.double()).float()).clamp(-127, 127)
    sums = codes.reshape(codes.shape[0], -1, GROUP).sum(dim=2)
    return codes.to(torch.int8), (t * r)[:, 0], sums.to(torch.int32), h


def _plain_rotate(x, c, s):
    half = x.shape[2] // 2
    a, b = x[:, :, :half].float(), x[:, :, half:].float()
    c, s = c[:, None], s[:, None]
    return torch.cat((a * c - b * s, b * c + a * s), dim=2).to(torch.bfloat16)


def _plain_append(state):
    offsets, lens, page = state["offsets"].long(), state["lens"].long(), state["k_cache"].shape[2]
    token = torch.arange(state["q"].shape[0], device=DEVICE)
    seq = (token[:, None] >= offsets[None, 1:]).sum(dim=1)
    position = lens[seq] - offsets[seq + 1] + token
    c, s = state["cos"][position], state["sin"][position]
    q, k = _plain_rotate(state["q"], c, s), _plain_rotate(state["k"], c, s)
    where = state["table"].long()[seq, position // page]
    state["k_cache"][where, :, position % page] = k
    state["v_cache"][where, :, position % page] = state["v"]
    return q, k, state["k_cache"], state["v_cache"]


def _plain_softmax(scores, seen):
    scores = torch.where(seen, scores, -torch.inf)
    p = torch.exp(scores - scores.amax(dim=-1, keepdim=True))
    return p / p.sum(dim=-1, keepdim=True)


def _plain_prompt(state):
    offsets, longest = state["offsets"].long(), state["longest"]
    q, k, v = state["q"].float(), state["k"].float(), state["v"].float()
    tokens, n_q, head = q.shape
    n_kv = k.shape[1]
    group, seqs = n_q // n_kv, offsets.numel() - 1
    place = torch.arange(longest, device=DEVICE)
    lens = offsets[1:] - offsets[:-1]
    index = (offsets[:-1, None] + place).clamp(max=tokens - 1)     # [sequences][longest], padded
    qb = q[index].reshape(seqs, longest, n_kv, group, head).permute(0, 2, 3, 1, 4).reshape(seqs, n_kv, group * longest, head).contiguous()
    kb = k[index].permute(0, 2, 3, 1).contiguous()
    vb = v[index].permute(0, 2, 1, 3).contiguous()
    scores = (qb @ kb).reshape(seqs, n_kv, group, longest, longest) * head ** -0.5
    # padded queries see what the last key sees; their rows are dropped
    p = _plain_softmax(scores, place[None, :] <= place[:, None])
    o = (p.reshape(seqs, n_kv, group * longest, longest) @ vb).reshape(seqs, n_q, longest, head).permute(0, 2, 1, 3)
    return o[place[None, :] < lens[:, None]].to(torch.bfloat16)


def _plain_decode(state):
    lens, table, page = state["lens"].long(), state["table"].long(), state["k_cache"].shape[2]
    q = state["q"].float()
    seqs, n_q, head = q.shape
    n_kv = state["k_cache"].shape[1]
    place = torch.arange(table.shape[1] * page, device=DEVICE)
    k = state["k_cache"][table].float().permute(0, 2, 4, 1, 3).reshape(seqs, n_kv, head, -1)
    v = state["v_cache"][table].float().permute(0, 2, 1, 3, 4).reshape(seqs, n_kv, -1, head)
    scores = (q.reshape(seqs, n_kv, n_q // n_kv, head) @ k) * head ** -0.5
    p = _plain_softmax(scores, (place[None, :] < lens[:, None])[:, None, None, :])
    return (p @ v).reshape(seqs, n_q, head).to(torch.bfloat16)


# ------------------------------------------------------------------ the work of a pass

def work(case):
    """Bytes and operations that one pass cannot do without."""
    if case["op"] in ("norm", "norm8"):
        n, rows = case["rows"] * case["hidden"], case["rows"]
        # x, residual and h; then y, or codes with their scale and sums
        out = 2 * n if case["op"] == "norm" else n + 4 * rows + 4 * n // GROUP
        return {"bytes": 6 * n + out + 2 * case["hidden"], "flops": (5 if case["op"] == "norm" else 8) * n}
    n_kv, n_q, head = case["n_kv"], case["n_kv"] * case["group"], case["head"]
    if case["op"] == "prompt":
        lengths = _lengths(case["seqs"], case["longest"], case["ragged"])
        pairs = sum(n * (n + 1) // 2 for n in lengths)
        return {"bytes": 2 * head * (2 * n_q + 2 * n_kv) * sum(lengths), "flops": 4 * head * n_q * pairs}
    new, lens = _cache_lens(case)
    if case["op"] == "append":
        tokens = sum(new)
        # q, k, v; q, k twice, v; and the angles of the positions, each read once
        return {"bytes": 2 * head * tokens * (2 * n_q + 5 * n_kv) + 4 * head * min(tokens, max(lens)), "flops": 3 * head * tokens * (n_q + n_kv)}
    keys = case["prefix"] + sum(n - case["prefix"] for n in lens)
    return {"bytes": 4 * head * n_kv * keys + 4 * head * n_q * case["seqs"], "flops": 4 * head * n_q * sum(lens)}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_attention(q, k, v, first):
    """q [n][group][head], k, v [keys][head], all of one key/value head; query i sees keys 0 .. first + i."""
    n, group, head = q.shape
    out = torch.empty(n, group, head, dtype=torch.float64, device=q.device)
    kt = k.double().t().contiguous()
    for at in range(0, n, 512):
        part = q[at:at + 512].double()
        seen = min(first + at + part.shape[0], k.shape[0])
        w = (part.reshape(-1, head) @ kt[:, :seen]).reshape(part.shape[0], group, seen) / head ** 0.5
        last = first + at + torch.arange(part.shape[0], device=q.device)
        w = w.masked_fill((torch.arange(seen, device=q.device) > last[:, None])[:, None], -torch.inf).softmax(dim=2)
        out[at:at + 512] = (w.reshape(-1, seen) @ v[:seen].double()).reshape(part.shape)
    return out


def exact(case, seed):
    """What `run` returns, from the definition in 64 bits."""
    inp = _inputs(case, seed)
    if case["op"] in ("norm", "norm8"):
        # the sum of two bf16 values is rounded to bf16 by the definition, and its 64-bit value is exact
        h = (inp["x"].double() + inp["residual"].double()).float().to(torch.bfloat16).double()
        rms = (h.square().mean(dim=1) + EPS).sqrt()
        if case["op"] == "norm":
            return h / rms[:, None] * inp["weight"].double(), h
        top = (h * inp["weight"].double()).abs().amax(dim=1)
        return None, top / 127.0 / rms, None, h
    n_kv, group, head = case["n_kv"], case["group"], case["head"]
    if case["op"] == "prompt":
        offsets = inp["offsets"].tolist()
        out = torch.empty(inp["q"].shape, dtype=torch.float64, device=DEVICE)
        for a, b in zip(offsets[:-1], offsets[1:]):
            for j in range(n_kv):
                heads = slice(j * group, (j + 1) * group)
                out[a:b, heads] = _exact_attention(inp["q"][a:b, heads], inp["k"][a:b, j], inp["v"][a:b, j], 0)
        return out
    lens, page = inp["lens"].tolist(), case["page"]
    if case["op"] == "append":
        k_cache, v_cache = inp["k_cache"].double(), inp["v_cache"].double()
        offsets = inp["offsets"].tolist()

        def turned(x, places):
            pairs = torch.complex(x[..., :head // 2].double(), x[..., head // 2:].double())
            turn = torch.complex(inp["cos"][places].double(), inp["sin"][places].double())
            y = pairs * turn[:, None]
            return torch.cat((y.real, y.imag), dim=2)

        q, k = [], []
        for b, n in enumerate(lens):
            t0, t1 = offsets[b], offsets[b + 1]
            places = torch.arange(n - (t1 - t0), n, device=DEVICE)
            q.append(turned(inp["q"][t0:t1], places))
            k.append(turned(inp["k"][t0:t1], places))
            at = inp["table"][b].long()[torch.div(places, page, rounding_mode="floor")]
            k_cache[at, :, places % page] = k[-1]
            v_cache[at, :, places % page] = inp["v"][t0:t1].double()
        return torch.cat(q), torch.cat(k), k_cache, v_cache
    out = torch.empty(inp["q"].shape, dtype=torch.float64, device=DEVICE)
    for b, n in enumerate(lens):
        used = inp["table"][b, :-(-n // page)].long()
        k = inp["k_cache"][used].transpose(0, 1).reshape(n_kv, -1, head)[:, :n]
        v = inp["v_cache"][used].transpose(0, 1).reshape(n_kv, -1, head)[:, :n]
        w = (inp["q"][b].double().reshape(n_kv, group, head) @ k.double().transpose(1, 2).contiguous()) / head ** 0.5
        out[b] = (w.softmax(dim=2) @ v.double()).reshape(-1, head)
    return out
