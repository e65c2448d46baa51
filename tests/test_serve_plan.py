"""The plan of single-token attention: its chunks cover the keys, stay within what the kernels hold, and the
workspace is what the size query says."""
import ctypes
import random

import pytest

import weight_only_int4_amd as w4
from tests.serve_plan import plan


def size_query(B, n_q, n_kv, head, page, max_len, prefix):
    size = ctypes.c_size_t(0)
    cache = w4._KVCache(None, None, 1, page, n_kv, head)
    rc = w4.load_library().w4_decode_attention(None, 0, B, n_q, ctypes.byref(cache), None, None, 0, max_len, prefix, 0.0, None, None,
                                               ctypes.byref(size), None)
    return size.value if rc == 0 else None


@pytest.mark.parametrize("seed", range(4))
def test_chunks_cover_the_keys(seed):
    rng = random.Random(seed)
    seen = set()
    for _ in range(3000):
        B, n_kv, group = int(2 ** rng.uniform(0, 10)), rng.choice((1, 2, 3, 8)), rng.choice((1, 3, 4, 7, 16, 24))
        head, page = rng.choice((64, 128)), rng.choice((16, 32, 64, 128, 256))
        max_len = int(2 ** rng.uniform(0, 18))
        prefix = rng.choice((0, page * rng.randrange(0, max_len // page + 2)))
        p = plan(B, n_kv * group, n_kv, head, page, max_len, prefix)
        seen.add(p.form)
        own = max_len - p.prefix
        assert p.group == group and p.prefix == (min(prefix, max_len) if B > 1 else 0) and p.rows == B * n_kv * group
        assert p.o_splits * p.o_chunk >= own and p.o_tiles * 16 >= group
        if p.direct:
            assert own <= 1024 and p.splits == 1 and p.bytes == 0
        else:
            assert p.o_chunk <= 1024 and p.o_chunk % 128 == 0 and (p.o_splits - 1) * p.o_chunk < max(own, 1)
            assert p.splits == p.p_splits + p.o_splits and p.bytes == p.stats_bytes + p.splits * p.rows * head * 4
        if p.prefix:
            assert p.p_chunk <= 1024 and p.p_chunk % 64 == 0 and p.p_splits * p.p_chunk >= p.prefix > (p.p_splits - 1) * p.p_chunk
            assert p.p_tiles * (128 if p.wide else 16) >= B * group
        assert size_query(B, n_kv * group, n_kv, head, page, max_len, prefix) in (p.bytes, None)
    assert seen == {"direct", "own", "prefix", "wide"}
