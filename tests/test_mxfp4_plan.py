"""Launch plans of the MXFP4 products, on the host: which kernels a call can reach."""
import re
import shutil
import subprocess

import pytest

import weight_only_int4_amd as w4
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
