"""Single-token attention by form (one launch; narrow chunks; narrow and shared prefix walks): what one form gives
for seen infinities, NaN and constant values the others give too.  The form of every case is pinned, so that a
rule that moves it to another one is noticed.  Tolerances as in test_gpu_serve.py."""
import math

import pytest
import torch

import weight_only_int4_amd as w4
from tests import test_gpu_serve as S
from tests.gpu_util import gpu_available, say
from tests.serve_plan import plan

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs an MI355X GPU")]

NAN, INF = float("nan"), float("inf")


def form_of(lens, n_q, n_kv, head, page, max_len, prefix):
    return plan(len(lens), n_q, n_kv, head, page, max_len, prefix)


# lens, prefix, max_len, the key whose value is not finite, the keys that lie low, form
LOW = [([280], 0, 280, 40, (32, 64), "direct"),                   # a wave's only tile
       ([280], 0, 2000, 40, (0, 128), "own"),                     # a chunk
       ([280], 0, 2000, 40, (32, 64), "own"),                     # a wave's tile of a chunk
       ([900, 33, 600], 0, 900, 700, (640, 768), "own"),
       ([270] * 4, 256, 270, 20, (0, 128), "prefix"),
       ([270] * 4, 256, 270, 264, (256, 270), "prefix"),          # the own tokens under a prefix
       ([4100] * 65, 4096, 4100, 300, (256, 512), "wide"),
       ([4100] * 65, 4096, 4100, 4097, (4096, 4100), "wide")]


@pytest.mark.parametrize("head", [64, 128])
@pytest.mark.parametrize("level", [-100.0, -400.0, -INF])
@pytest.mark.parametrize("lens,prefix,max_len,at,low,form", LOW)
def test_values_of_keys_that_weigh_nothing(head, level, lens, prefix, max_len, at, low, form):
    """An infinity or NaN in a value that a sequence sees is not lost where its weight underflows to 0, or is 0 for a
    score of -infinity: 0 times it is NaN, whichever way the keys are cut.  (A weight that a form keeps above 0 gives
    the infinity.)  Its other channels are the others' keys alone."""
    page, n_kv, n_q = 16, 2, 8 if head == 128 else 16
    say("low", form, head, level, lens[:2], at)
    assert form_of(lens, n_q, n_kv, head, page, max_len, prefix).form == form
    for seed, what in enumerate((NAN, INF, -INF)):
        gen = S.generator(seed)
        kc, vc, table, keys, values = S.paged(gen, lens, n_kv, head, page, prefix)
        table = torch.nn.functional.pad(table, (0, max(0, -(-max_len // page) - table.shape[1])), value=-1)
        q = S.fused(gen, len(lens), n_q, n_kv, head)[0].clone()
        q[:, :, 0] = 8
        shared = at < prefix
        rows = range(len(lens)) if shared else [0]
        k0 = level * head ** 0.5 / 8
        for p in range(*low):
            kc[int(table[0, p // page]), :, p % page, 0] = k0
        vc[int(table[0, at // page]), :, at % page, 5] = what
        for b in rows:
            kept = torch.ones(lens[b], dtype=torch.bool, device="cuda")
            kept[low[0]:low[1]] = False                            # below the others by 100: they weigh e^-90 at most
            keys[b], values[b] = keys[b][kept], values[b][kept]
        o = w4.decode_attention(q, kc, vc, S.ints(lens), table, max_len=max_len, prefix_len=prefix)
        hit = o[list(rows), :, 5].float()
        assert torch.isnan(hit).all() if math.isnan(what) else (torch.isnan(hit) | (hit == what)).all()
        plain, zeroed = o.clone(), [v.clone() for v in values]
        for b in rows:
            plain[b, :, 5] = 0
            zeroed[b][:, :, 5] = 0
        S.check_decode(plain, q, keys, zeroed, head ** -0.5)
        if lens[0] <= 300:                                         # the one-launch form of sequence 0 by itself
            assert form_of(lens[:1], n_q, n_kv, head, page, lens[0], 0).form == "direct"
            alone = w4.decode_attention(q[:1], kc, vc, S.ints(lens[:1]), table[:1], max_len=lens[0])
            assert S.same_bits(o[:1], alone)


# n_q, n_kv, lens, prefix, form
CONSTANT = [(4, 2, [300], 0, "direct"), (4, 2, [1200, 900, 0, 1], 0, "own"), (16, 2, [700] * 9, 512, "prefix"), (32, 4, [2100] * 65, 2048, "wide")]


@pytest.mark.parametrize("head", [64, 128])
@pytest.mark.parametrize("n_q,n_kv,lens,prefix,form", CONSTANT)
def test_constant_values_come_back(head, n_q, n_kv, lens, prefix, form):
    """Values that are the same in every key are the output, to the bit: the weights are summed as they are multiplied.
    (Weights of 0.5018 round to 0.5: summed unrounded they would take 0.3% off.)  n additions in fp32 and the joins
    are off by 2 n 2^-23 <= 2^-10 here, less than the half step (2^-9) that a bf16 value bears."""
    if head == 64:
        n_q *= 2
    assert max(lens) <= 4096 and form_of(lens, n_q, n_kv, head, 16, max(lens), prefix).form == form
    gen = S.generator(head)
    kc, vc, table, keys, values = S.paged(gen, lens, n_kv, head, 16, prefix, stale=0)
    u = torch.randn(n_kv, head, generator=gen, device="cuda").to(S.BF)
    kc[:, :, :, 0] = -1
    kc[:, :, ::16, 0] = 0                                          # one key of every tile on top
    kc[:, :, :, 1:] = 0
    vc[:] = u[None, :, None]
    q = torch.zeros(len(lens), n_q, head, dtype=S.BF, device="cuda")
    q[:, :, 0] = 1
    o = w4.decode_attention(q, kc, vc, S.ints(lens), table, max_len=max(lens), prefix_len=prefix, scale=-math.log(0.5018))
    want = u.repeat_interleave(n_q // n_kv, 0)
    for b, n in enumerate(lens):
        assert S.same_bits(o[b], want if n else torch.zeros_like(want))
    if form == "direct":                                           # the prompt's form, whose sums have always been these
        p = w4.prompt_attention(q.expand(300, n_q, head).contiguous(), kc[0, 0, 0].expand(300, n_kv, head).contiguous(),
                                u.expand(300, n_kv, head).contiguous(), S.ints([0, 300]))
        assert S.same_bits(p, want.expand(300, n_q, head))


def spread_lengths(prefix, longest, count):
    """Lengths at and between the borders of tiles, chunks and the prefix, `count` of them; the first reaches past the prefix."""
    some = [longest, 0, 1, 15, 16, 17, 63, 64, 65, 255, 256, 257, 300, prefix - 17, prefix - 16, prefix - 1, prefix, prefix + 1, prefix + 130]
    return (some + [(37 * i * i + 11 * i) % (longest + 1) for i in range(count)])[:count]


# head, n_q, n_kv, page, prefix, longest, sequences, keys of a chunk
WIDE = [(128, 8, 2, 16, 4112, 4500, 67, 256),                      # the last chunk is 16 keys, rows 268
        (64, 16, 2, 16, 4112, 4500, 67, 256),
        (128, 6, 2, 32, 5472, 5472, 67, 256),                      # nothing behind the prefix, group 3
        (64, 14, 2, 64, 4736, 4900, 70, 256),                      # group 7
        (64, 32, 1, 256, 8448, 8700, 70, 640),                     # one key/value head, pages of 256
        (128, 8, 2, 16, 16400, 16500, 65, 384),                    # chunks of another length; the last is short
        (128, 32, 8, 64, 2304, 4600, 64, 1024),                    # long chunks: 64 pages in a wave
        (64, 64, 8, 16, 2320, 6400, 64, 1024)]


@pytest.mark.parametrize("head,n_q,n_kv,page,prefix,longest,count,chunk", WIDE)
def test_shared_prefix_walk(head, n_q, n_kv, page, prefix, longest, count, chunk):
    say("wide", head, n_q, n_kv, page, prefix, longest)
    lens = spread_lengths(prefix, longest, count)
    p = form_of(lens, n_q, n_kv, head, page, longest, prefix)
    assert p.form == "wide" and p.p_chunk == chunk
    gen = S.generator(prefix + head)
    kc, vc, table, keys, values = S.paged(gen, lens, n_kv, head, page, prefix)
    q = S.fused(gen, count, n_q, n_kv, head)[0]
    o = w4.decode_attention(q, kc, vc, S.ints(lens), table, max_len=longest, prefix_len=prefix)
    some = range(count) if n_kv < 8 else range(0, count, 5)        # (the 64-bit attention of all would take a minute)
    S.check_decode(o[list(some)], q[list(some)], [keys[b][:longest] for b in some], [values[b][:longest] for b in some], head ** -0.5)
    assert not o[1].any()
    assert S.same_bits(o, w4.decode_attention(q, kc, vc, S.ints(lens), table, max_len=longest, prefix_len=prefix))


@pytest.mark.parametrize("head,n_q", [(64, 16), (128, 8)])
def test_shared_prefix_walk_cut_by_max_len(head, n_q):
    """max_len inside the prefix, in the middle of a page: tokens from there on are left out."""
    prefix, cut, n_kv = 8192, 4501, 2
    lens = spread_lengths(prefix, 8300, 67)
    p = form_of(lens, n_q, n_kv, head, 16, cut, prefix)
    assert p.form == "wide" and p.prefix == cut and p.o_splits == 0
    gen = S.generator(head)
    kc, vc, table, keys, values = S.paged(gen, lens, n_kv, head, 16, prefix)
    q = S.fused(gen, len(lens), n_q, n_kv, head)[0]
    o = w4.decode_attention(q, kc, vc, S.ints(lens), table, max_len=cut, prefix_len=prefix)
    S.check_decode(o, q, [k[:cut] for k in keys], [v[:cut] for v in values], head ** -0.5)


@pytest.mark.parametrize("head,n_q", [(64, 16), (128, 8)])
def test_shared_prefix_walk_leaves_out_bad_pages(head, n_q):
    prefix, n_kv, page = 4112, 2, 16
    lens = spread_lengths(prefix, 4500, 67)
    assert form_of(lens, n_q, n_kv, head, page, 4500, prefix).form == "wide"
    gen = S.generator(head + 1)
    kc, vc, table, keys, values = S.paged(gen, lens, n_kv, head, page, prefix)
    q = S.fused(gen, len(lens), n_q, n_kv, head)[0]
    kept = torch.ones(prefix, dtype=torch.bool, device="cuda")
    gone = list(zip((0, 3, 17, 18, 19, 100, 255, 256), (-1, 2 ** 31 - 1, -2 ** 31, len(kc), 10 ** 9, -7, len(kc) + 1, -1)))
    gone += [(i, -1) for i in range(32, 52)]                        # a whole chunk, and some of the next
    for i, bad in gone:
        table[0, i] = bad
        kept[16 * i:16 * i + 16] = False
    pick = lambda t: torch.cat((t[:prefix][kept[:len(t)]], t[prefix:]))  # noqa: E731
    o = w4.decode_attention(q, kc, vc, S.ints(lens), table, max_len=4500, prefix_len=prefix)
    S.check_decode(o, q, [pick(k) for k in keys], [pick(v) for v in values], head ** -0.5)


@pytest.mark.parametrize("head,n_q", [(64, 16), (128, 8)])
def test_shared_prefix_walk_short_rows_under_nan(head, n_q):
    """NaN in a prefix token's value reaches the sequences that see it, in its channel, and no other."""
    prefix, n_kv, page, at = 4112, 2, 16, 2000
    lens = spread_lengths(prefix, 4500, 67)
    assert form_of(lens, n_q, n_kv, head, page, 4500, prefix).form == "wide"
    gen = S.generator(head + 2)
    kc, vc, table, keys, values = S.paged(gen, lens, n_kv, head, page, prefix)
    q = S.fused(gen, len(lens), n_q, n_kv, head)[0]
    vc[int(table[0, at // page]), :, at % page, 7] = NAN
    o = w4.decode_attention(q, kc, vc, S.ints(lens), table, max_len=4500, prefix_len=prefix)
    sees = torch.tensor([n > at for n in lens], device="cuda")
    assert torch.isnan(o[sees][:, :, 7].float()).all()
    o[sees, :, 7] = 0
    for b in range(len(lens)):
        if lens[b] > at:
            values[b] = values[b].clone()
            values[b][:, :, 7] = 0
    S.check_decode(o, q, keys, values, head ** -0.5)


@pytest.mark.parametrize("head,n_q", [(64, 16), (128, 8)])
def test_shared_prefix_walk_past_32_bits(head, n_q):
    """The prefix's pages past 2^32 bytes of the cache: the same as in a small one."""
    prefix, n_kv, page = 4352, 2, 64
    lens = [prefix + 5 * i for i in range(65)]
    assert form_of(lens, n_q, n_kv, head, page, max(lens), prefix).form == "wide"
    gen = S.generator(head + 3)
    small_k, small_v, small_table, keys, values = S.paged(gen, lens, n_kv, head, page, prefix)
    pages = (5 << 30) // (n_kv * page * head * 2)
    kc = torch.empty(pages, n_kv, page, head, dtype=S.BF, device="cuda")
    vc = torch.empty_like(kc)
    kc[-len(small_k):], vc[-len(small_v):] = small_k, small_v
    ok = (small_table >= 0) & (small_table < len(small_k))
    table = torch.where(ok, small_table + (pages - len(small_k)), small_table)
    q = S.fused(gen, len(lens), n_q, n_kv, head)[0]
    o = w4.decode_attention(q, kc, vc, S.ints(lens), table, max_len=max(lens), prefix_len=prefix)
    assert S.same_bits(o, w4.decode_attention(q, small_k, small_v, S.ints(lens), small_table, max_len=max(lens), prefix_len=prefix))
    S.check_decode(o, q, keys, values, head ** -0.5)
