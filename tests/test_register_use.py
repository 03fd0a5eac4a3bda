"""Registers of the stream-K kernels: the epilogue they share with the product with
scales must not make an instance spill more than it did without it."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CSRC = os.path.join(ROOT, "matrix_core_gemm_amd", "csrc")


def spilled(tmp_path, op, args, la, lb):
    """Vector registers that the 256 x 256 stream-K instance of gemm_fast_kernel spills."""
    src = tmp_path / "instance.hip"
    src.write_text(f'#include "gemm_fast_kernel.hpp"\nnamespace mcg {{\nhipError_t instance(const {args}& a, hipStream_t s) '
                   f"{{ return fast::launch_one<fast::{op}, {la}, {lb}, 256, true>(a, s); }}\n}}\n")
    # (as build.py compiles them)
    p = subprocess.run([HIPCC, "-x", "hip", "-O3", "-std=c++17", "-fPIC", "--offload-arch=gfx950", "-Xclang", "-target-feature",
                        "-Xclang", "-packed-fp32-ops", "--cuda-device-only", "-Rpass-analysis=kernel-resource-usage", "-I" + CSRC,
                        "-c", str(src), "-o", str(tmp_path / "instance.o")], capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stderr
    found = {}
    for block in p.stderr.split("Function Name: ")[1:]:
        name = block.split()[0]
        if "gemm_fast_kernel" in name and "Li256ELb1E" in name:
            found[name] = int(re.search(r"VGPRs Spill: (\d+)", block)[1])
    assert len(found) == 1, found
    return found.popitem()[1]


@pytest.mark.skipif(shutil.which(HIPCC) is None, reason="no hipcc")
@pytest.mark.parametrize("op,args,la,lb,most", [
    ("I8", "DenseArgs", "LAYOUT_K", "LAYOUT_K", 80),
    ("BF16", "DenseArgs", "LAYOUT_K", "LAYOUT_K", 66),
    ("I8Scaled", "ScaledArgs", "LAYOUT_K", "LAYOUT_K", 55),
])
def test_stream_k_instances_spill_no_more_than_they_did(tmp_path, op, args, la, lb, most):
    assert spilled(tmp_path, op, args, la, lb) <= most
