"""Where a workgroup of a product by group finds its rows (csrc/group_tiles.hpp), on the
host: whatever the offsets hold, a group's rows lie inside the operand, and valid
offsets give their rows; the tile order of the 8 XCDs takes every tile once."""
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
SOURCE = """
#include <stdint.h>
#include "group_tiles.hpp"
extern "C" void rows(const int32_t* offsets, int groups, int64_t M, int64_t* out) {
  for (int g = 0; g < groups; ++g) {
    const mcg::GroupRows r = mcg::group_rows(offsets, g, M);
    out[2 * g] = r.r0;
    out[2 * g + 1] = r.r1;
  }
}
extern "C" int order(int bid, int n) { return mcg::xcd_order(bid, n); }
"""

pytestmark = pytest.mark.skipif(shutil.which(HIPCC) is None, reason="no hipcc")


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    import ctypes
    d = tmp_path_factory.mktemp("group_tiles")
    (d / "a.hip").write_text(SOURCE)
    subprocess.check_call([HIPCC, "-x", "hip", "-O1", "-std=c++17", "-fPIC", "-shared", "--cuda-host-only", "--offload-arch=gfx950",
                           "-I" + os.path.join(ROOT, "matrix_core_gemm_amd", "csrc"), str(d / "a.hip"), "-o", str(d / "a.so")])
    return ctypes.CDLL(str(d / "a.so"))


def rows(lib, offsets, M):
    import ctypes
    n = len(offsets) - 1
    out = (ctypes.c_int64 * (2 * n))()
    lib.rows((ctypes.c_int32 * (n + 1))(*offsets), n, ctypes.c_int64(M), out)
    return [(out[2 * i], out[2 * i + 1]) for i in range(n)]


def test_valid_offsets_give_their_rows(lib):
    off = [2, 2, 7, 7, 30, 31]
    assert rows(lib, off, 31) == list(zip(off, off[1:]))
    assert rows(lib, [0, 0], 0) == [(0, 0)]


def test_no_offsets_leave_the_operand(lib):
    rng = random.Random(5)
    extreme = [-2 ** 31, -1, 0, 1, 99, 100, 101, 2 ** 31 - 1]
    for M in (0, 1, 100, 2 ** 31 - 1):
        for _ in range(500):
            for r0, r1 in rows(lib, [rng.choice(extreme + [rng.randrange(-200, 300)]) for _ in range(9)], M):
                assert 0 <= r0 <= r1 <= M


@pytest.mark.parametrize("n", [1, 7, 8, 9, 63, 64, 1000, 4099])
def test_the_xcd_order_takes_every_tile_once(lib, n):
    seen = [lib.order(b, n) for b in range(n)]
    assert sorted(seen) == list(range(n))
    # workgroups of one XCD (every eighth) take consecutive tiles
    for x in range(min(8, n)):
        mine = seen[x::8]
        assert mine == list(range(mine[0], mine[0] + len(mine)))
