"""The choice of a kernel by the products by group and of block-scaled 8-bit floats (host
only: 256 compute units where no device is visible), and what their kernels keep in
registers."""
import os
import shutil

import pytest

import experts_cases as cases
from test_register_use import CSRC, HIPCC, spills

m = pytest.importorskip("matrix_core_gemm_amd")
FAKE = 1 << 20  # aligned; never read


@pytest.mark.parametrize("name", list(cases.GROUPED))
def test_grouped_cases_take_their_form(name):
    case = cases.GROUPED[name]
    dt, dtD, lb, sizes, N, K, pad, kernel, tile = case
    G, M, lda, ldb, strideB = cases.operands_of_grouped(case)
    assert m.grouped_path(dt, "k_contig", lb, G, M, N, K, FAKE, lda, FAKE, ldb, strideB, 128, dtD) == (kernel, tile)


@pytest.mark.parametrize("name", list(cases.GRAD))
def test_grouped_grad_cases_take_their_form(name):
    dt, dtD, sizes, M, N, pad, kernel, tile = cases.GRAD[name]
    assert m.grouped_grad_path(dt, len(sizes), M, N, sum(sizes), FAKE, M + pad, FAKE, N + pad, dtD) == (kernel, tile)


@pytest.mark.parametrize("name", list(cases.F8))
def test_f8_cases_take_their_form(name):
    to, dtD, la, lb, bb, M, N, K, pad, kernel, tile = cases.F8[name]
    lda, ldb = (K if la == "k_contig" else M) + pad, (K if lb == "k_contig" else N) + pad
    assert m.grouped_path(to, la, lb, 0, M, N, K, FAKE, lda, FAKE, ldb, 0, bb, dtD) == (kernel, tile)


@pytest.mark.parametrize("dt,dtD", [("bf16", "bf16"), ("e4m3", "bf16"), ("e4m3", "f32")])
@pytest.mark.parametrize("change", [dict(A=FAKE + 8), dict(B=FAKE + 8), dict(lda=4104 - 4), dict(ldb=4104 - 4), dict(strideB=4096 * 4096 + 4),
                                    dict(K=4090), dict(lda=1 << 24)], ids=str)
def test_operands_without_16_byte_rows_take_the_general_kernel(dt, dtD, change):
    a = dict(A=FAKE, lda=4096, B=FAKE, ldb=4096, strideB=4096 * 4096, K=4096)
    call = lambda a: m.grouped_path(dt, "k_contig", "k_contig", 8, 8192, 4096, a["K"], a["A"], a["lda"], a["B"], a["ldb"], a["strideB"], 128, dtD)
    assert call(a)[0] != cases.GENERAL
    assert call({**a, **change})[0] == cases.GENERAL


def test_kinds_that_the_pipelined_8_bit_kernel_lacks_take_the_general_one():
    for la, lb, bb in (("k_contig", "k_contig", 1), ("k_contig", "mn_contig", 1), ("mn_contig", "k_contig", 128), ("mn_contig", "k_contig", 1),
                       ("mn_contig", "mn_contig", 128)):
        assert m.grouped_path("e4m3", la, lb, 0, 4096, 4096, 4096, FAKE, 4096, FAKE, 4096, 0, bb, "bf16")[0] == cases.GENERAL


def test_the_choice_follows_the_work():
    def tile(M, G=0, N=4096, K=4096, dtD="bf16", dt="e4m3"):
        return m.grouped_path(dt, "k_contig", "k_contig", G, M, N, K, FAKE, K, FAKE, K, N * K, 128, dtD)
    assert tile(1) == (cases.FEW, 16) and tile(8192) == (cases.PIPE_256, 256)
    assert tile(500) == (cases.PIPE_64, 64)
    assert tile(8192, dtD="f32")[1] in (64, 128)   # exact products: no 256 x 256 form
    assert m.grouped_path("e4m3", "mn_contig", "mn_contig", 0, 8192, 8192, 8192, FAKE, 8192, FAKE, 8192, 0, 1, "bf16") == (cases.PIPE_128, 128)
    assert tile(8192, G=16, dt="bf16") == (cases.PIPE_256, 256)
    assert tile(32, G=16, dt="bf16") == (cases.FEW, 16)
    for M in (1, 7, 33, 64, 65, 1000, 4097):
        for G in (0, 1, 8, 64, 4096, 65535):
            kernel, rows = tile(M, G)
            assert kernel in (cases.FEW, cases.PIPE_64, cases.PIPE_128, cases.PIPE_256) and rows in (16, 32, 64, 128, 256)


def test_a_launch_holds_the_tiles_of_the_choice():
    """At the most rows, groups and columns that a call may have, and just below: fewer than 2^23 workgroups."""
    for dt, dtD, most in (("bf16", "bf16", 128), ("e4m3", "bf16", 64), ("e4m3", "f32", 64)):
        for G, M in ((65535, 65535), (65535, 200000), (65535, 1 << 22), (1000, 1000), (0, 64), (0, 1 << 20), (8, 1 << 25)):
            def tiles(t):
                some = min(max(G, 1), M)
                return -(-M // t) if G == 0 else (M - some) // t + some
            cols = (2**23 - 65) // tiles(most)
            for N in (128 * cols, 64 * cols, 32 * cols, 128 * cols // 5 * 4 + 1):
                if not 0 < N < 1 << 24:
                    continue
                for K in (16, 128, 1024):
                    kernel, rows = m.grouped_path(dt, "k_contig", "k_contig", G, M, N, K, FAKE, K, FAKE, K, N * K, 128, dtD)
                    assert kernel >= 0, (dt, G, M, N, K)
                    if kernel != cases.TINY:
                        wide = {cases.FEW: 32, cases.PIPE_256: 256}.get(kernel, 128)
                        assert tiles(rows) * -(-N // wide) < 2**23, (dt, G, M, N, K, kernel, rows)
            assert m.grouped_path(dt, "k_contig", "k_contig", G, M, 128 * cols + 1, 128, FAKE, 128, FAKE, 128, 0, 128, dtD)[0] == -1


@pytest.mark.skipif(shutil.which(HIPCC) is None, reason="no hipcc")
@pytest.mark.parametrize("source", ["blocks_quant.hip", "expert_rows.hip", "f8_blocks.hip"])
def test_kernels_that_spill_nothing(tmp_path, source):
    found = spills(tmp_path, os.path.join(CSRC, source))
    assert len(found) >= 4 and not any(found.values()), {k: n for k, n in found.items() if n}
