"""Build libw4a16.so (HIP, gfx950) in-tree with hipcc.

    python -m weight_only_int4_amd.build [--jobs N]

Every .hip file under csrc/ is compiled to an object in ``_build/`` at the repo
root and linked into ``weight_only_int4_amd/libw4a16.so``.  Floating point stays
IEEE (no fast-math; correctly rounded fp32 division is hipcc's default).  Packed
fp32 instructions are disabled for all device code.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libw4a16.so")
ARCH = "gfx950"

HIPCC_FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-Wall",
    "-Wno-unused-function",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
]


# keep MFMA accumulators in ordinary VGPRs: the int4 GEMM folds them with VALU
# FMAs every group, and accumulator-register copies would double its VALU work
VGPR_ACC_FLAGS = ["-mllvm", "-amdgpu-mfma-vgpr-form=1"]
# kernels that never touch their accumulators between MFMAs, and need all 512 registers
# of one wave per SIMD
ACC_REGISTER_SOURCES = {"mxfp4_gemm.hip"}


# the library links nothing beyond the HIP runtime
LINK_LIBS: list[str] = []


def hipcc() -> str:
    path = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(path):
        raise RuntimeError("hipcc not found: the W4A16 library needs ROCm's hipcc to build")
    return path


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".hip"))


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    form = [] if os.path.basename(src) in ACC_REGISTER_SOURCES else VGPR_ACC_FLAGS
    cmd = [hipcc(), *HIPCC_FLAGS, *form, "-c", src, "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{res.stdout}\n{res.stderr}")
    return obj


def build(jobs: int | None = None, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sources()
    jobs = jobs or min(len(srcs), max(1, (os.cpu_count() or 4) // 2), 8)
    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        objs = list(ex.map(_compile, srcs))
    tmp = LIB + ".tmp"
    cmd = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs, *LINK_LIBS]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB} from {len(srcs)} sources")
    return LIB


def main(argv=None) -> int:
    ap = argparse.ArgumentParser()
    ap.add_argument("--jobs", type=int, default=None)
    args = ap.parse_args(argv)
    build(args.jobs, verbose=True)
    return 0


if __name__ == "__main__":
    sys.exit(main())
