"""Launch plans of the MXFP4 products, on the host: which kernels a call can reach."""
import ctypes
import re
import shutil
import subprocess

import pytest

import weight_only_int4_amd as w4
from tests import mx_forms
from tests.mx_plan import plan, random_shapes


def _compiled_stream_kernels():
    nm = shutil.which("nm")
    if nm is None:
        pytest.skip("needs nm")
    out = subprocess.run([nm, "-C", w4.library_path()], capture_output=True, text=True, check=True).stdout
    found = set(re.findall(r"__device_stub__mx_stream_kernel<(\d+), (\d+), (\d+), (\d+)>", out))
    if not found:
        pytest.skip("the library has no local symbols")
    return {tuple(map(int, f)) for f in found}


def test_every_compiled_stream_kernel_is_planned():
    """(activation bits, slices, row tiles, channel tiles): no instance that no shape takes, none that is missing."""
    reached = set()
    for act, M, K, N in random_shapes(150_000, 1):
        p = plan(act, M, K, N)
        if p and p[0] == "stream":
            reached.add((act,) + p[1:4])
    compiled = _compiled_stream_kernels()
    assert compiled - reached == set()
    assert reached - compiled == set()


def test_listed_shapes_take_the_plans_they_stand_for():
    """A changed rule must not move the GPU tests off a kernel unseen."""
    for act, M, K, N, want in mx_forms.STREAM + mx_forms.TILE:
        assert plan(act, M, K, N)[1:] == want, (act, M, K, N)
        assert plan(act, M, K, N)[0] == ("stream" if (act, M, K, N, want) in mx_forms.STREAM else "tile")


def test_every_planned_kernel_has_a_gpu_test():
    """Kernel instances (and, per instance, K split or not, and padded scale rows) against the shapes that the GPU
    tests run."""
    from tests import test_gpu_mxfp4 as g
    tested = {_kind(act, *s) for act in (16, 4) for s in g.SMALL + g.MEDIUM + g.LARGE + g.TILED + g.STREAM}
    tested |= {_kind(*s[:4]) for s in mx_forms.STREAM + mx_forms.TILE}
    # of shapes that a test runs in seconds
    reached = {_kind(*s) for s in random_shapes(150_000, 2) if s[1] * s[2] * s[3] <= 2e11 and s[2] * max(s[1], s[3]) <= 1e8}
    assert reached - tested == set()


def _kind(act, M, K, N):
    p = plan(act, M, K, N)
    return p and (act,) + tuple(x > 1 if i == len(p) - 1 and p[0] == "stream" or i == 2 and p[0] == "tile" else x
                                for i, x in enumerate(p))


def test_workspace_needs():
    """What the size query says: scale rows that need padding, or K split over workgroups, and nothing else."""
    lib = w4.load_library()
    for act, fn, nulls in ((16, lib.mxfp4_a16_gemm, 1), (4, lib.mxfp4_a4_gemm, 2)):
        for M, K, N in ((1, 2048, 2048), (16, 17408, 512), (64, 17408, 64), (200, 17408, 128), (2048, 2048, 6144),
                        (37, 6176, 2047), (513, 2016, 2050), (40, 17408, 1500), (65, 8192, 9001)):
            sz = ctypes.c_size_t(12345)
            assert fn(*[None] * nulls, M, K, N, None, None, None, None, ctypes.byref(sz), None) == 0
            p = plan(act, M, K, N)
            split = p[4] if p[0] == "stream" else p[2]
            partials = 4 * split * M * N if split > 1 else 0
            blocks = (K // 32 + 3) // 4 * 4
            pads = (N * blocks + (M * blocks if act == 4 else 0)) if p[0] == "tile" and p[4] else 0
            assert partials + pads <= sz.value <= partials + pads + 512, (act, M, K, N)
            assert (sz.value > 0) == (split > 1 or pads > 0)
