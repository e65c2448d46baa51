"""What precedes a copy to LDS in the listing of a kernel built here: a vector instruction that writes a scalar
register needs five wait states before a memory instruction reads it, and the compiler does not look into inline asm."""
import re
import shutil
import subprocess

import pytest

from weight_only_int4_amd import build

SOURCE = """
#include "flash_tile.hpp"
using namespace w4;
__global__ void copies(uint32_t high, const uint32_t* shift, uint32_t* out) {{
  extern __shared__ uint32_t lds[];
  const uint32_t at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)lds;
  const uint32_t low = __builtin_amdgcn_readfirstlane(shift[threadIdx.x]);    // by a vector instruction, right before
  {copy}(threadIdx.x * 16, reinterpret_cast<const void*>((uint64_t)high << 32 | low), at);
  wait_vmcnt<0>();
  __syncthreads();
  out[threadIdx.x] = lds[threadIdx.x];
}}
"""


def scalar_registers(text):
    """The numbers of the scalar registers that an operand list names."""
    out = set()
    for first, last in re.findall(r"\bs\[(\d+):(\d+)\]", text):
        out |= set(range(int(first), int(last) + 1))
    return out | {int(n) for n in re.findall(r"\bs(\d+)\b", text)}


def wait_states(lines):
    """For each copy to LDS: the wait states since a vector instruction wrote its base, or None where the last to write it
    was a scalar instruction (which needs none) or nothing."""
    found = []
    for i, line in enumerate(lines):
        if not line.startswith("global_load_lds"):
            continue
        base, states, result = scalar_registers(line), 0, None
        for before in reversed(lines[:i]):
            op, _, rest = before.partition(" ")
            if base & scalar_registers(rest.split(",")[0]) and op.startswith(("v_", "s_")):
                base -= scalar_registers(rest.split(",")[0])
                if op.startswith("v_"):
                    result = states
                if result is not None or not base:
                    break
            states += int(rest, 0) + 1 if op == "s_nop" else 1
        found.append(result)
    return found


@pytest.mark.skipif(shutil.which("hipcc") is None, reason="needs hipcc")
@pytest.mark.parametrize("copy", ["lds_copy16", "lds_copy4", "lds_copy16_free"])
def test_a_copys_base_is_waited_for(copy, tmp_path):
    src, out = tmp_path / "copies.hip", tmp_path / "copies.s"
    src.write_text(SOURCE.format(copy=copy))
    res = subprocess.run([build.hipcc(), *build.HIPCC_FLAGS, "-I", build.CSRC, "-S", "--cuda-device-only", str(src), "-o", str(out)],
                         capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    lines = [t.split(";")[0].strip().replace("\t", " ") for t in out.read_text().splitlines()]
    lines = [t for t in lines if t and not t.startswith((".", "/")) and not t.endswith(":")]
    states = wait_states(lines)
    assert any(t.startswith("v_readfirstlane") for t in lines)     # the base is a vector instruction's
    assert len(states) == 1 and (states[0] is None or states[0] >= 5), states
