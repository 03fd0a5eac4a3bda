"""Plans of the 8-bit products on the host: the kernel, panels and workspace that a call
takes (mcg_i8_scaled_path, mcg_grad_i8_path)."""
import pytest

import linear8_cases as cases
import linear8_ref as ref

m = pytest.importorskip("matrix_core_gemm_amd")

BASE = 0x10000  # aligned and non-null; never dereferenced here
FREE = 1 << 50  # a workspace without a limit
GENERAL, FAST, STREAM, MID, HALF, TINY = 0, 1, 4, 6, 7, 16


def up(x, y):
    return -(-x // y) * y


@pytest.mark.parametrize("layout,M,N,K", [("k_contig", 465, 67138, 35788), ("mn_contig", 568, 46796, 50172)])
def test_scaled_workspace_covers_the_last_panel(layout, M, N, K):
    # panels below 2 GiB each; the last, narrower one takes more stream-K slots than the others
    lda, ldb = K + 1, (K if layout == "k_contig" else N) + 1
    need = m.i8_scaled_workspace_bytes(layout, M, N, K, BASE, lda, BASE, ldb)
    kernel, plan = m.i8_scaled_path(layout, M, N, K, BASE, lda, BASE, ldb, FREE)
    pn, kp = plan["panel"], up(K, 16)
    assert kernel in (FAST, MID) and 0 < pn < N and plan["workspace"] == need
    last = N - (-(-N // pn) - 1) * pn
    slots = [m.i8_scaled_path(layout, M, n, kp, BASE, kp, BASE, kp if layout == "k_contig" else up(pn, 16), FREE)[1]["workspace"]
             for n in (pn, last)]  # of the products on the copies
    copies = M * kp + kp * (pn if layout == "k_contig" else up(pn, 16))
    assert slots[1] > slots[0] and need == copies + slots[1]
    assert m.i8_scaled_path(layout, M, N, K, BASE, lda, BASE, ldb, need) == (kernel, plan)


@pytest.mark.parametrize("layout,M,N,K", [("k_contig", 408, 66576, 16336), ("mn_contig", 456, 12848, 85712)])
def test_gradient_workspace_covers_the_last_panel(layout, M, N, K):
    lda = K if layout == "k_contig" else M
    need = m.grad_i8_workspace_bytes("bf16", layout, M, N, K, BASE, lda, BASE, N, "bf16")
    kernel, plan = m.grad_i8_path("bf16", layout, M, N, K, BASE, lda, BASE, N, "bf16", FREE)
    pn = plan["panel"]
    assert kernel in (FAST, MID) and 0 < pn < N and plan["workspace"] == need
    last = N - (-(-N // pn) - 1) * pn
    slots = []
    for n in (pn, last):
        p = m.grad_i8_path("bf16", layout, M, n, K, BASE, lda, BASE, N, "bf16", FREE)[1]
        assert p["panel"] == n
        slots.append(p["workspace"] - K * up(n, 16) * 2)
    assert slots[1] > slots[0] and need == K * pn * 2 + slots[1]
    assert m.grad_i8_path("bf16", layout, M, N, K, BASE, lda, BASE, N, "bf16", need) == (kernel, plan)


def test_a_plan_keeps_to_its_workspace():
    for ws in (0, 16, 1 << 16, 1 << 20, 9 << 20, 40 << 20, FREE):
        for M, N, K in ((1, 4096, 4096), (24, 4096, 16384), (93, 1216, 8128), (700, 1500, 3001), (3000, 2000, 4096), (5, 3, 2)):
            for layout in ("k_contig", "mn_contig"):
                ldb = K if layout == "k_contig" else N
                _, p = m.i8_scaled_path(layout, M, N, K, BASE, K, BASE, ldb, ws)
                assert 0 <= p["workspace"] <= ws and p["ranges"] >= 1 and p["panel"] <= N
                for dt in ("bf16", "f32"):
                    _, p = m.grad_i8_path("bf16", layout, M, N, K, BASE, K if layout == "k_contig" else M, BASE, N, dt, ws)
                    assert 0 <= p["workspace"] <= ws and p["ranges"] >= 1 and p["panel"] <= N


def test_paths_of_refused_and_empty_products():
    assert m.i8_scaled_path("k_contig", 0, 8, 8, BASE, 8, BASE, 8, FREE)[0] == -1
    assert m.i8_scaled_path("k_contig", 8, 8, 200000, BASE, 200000, BASE, 200000, FREE)[0] == -1
    assert m.i8_scaled_path(2, 8, 8, 8, BASE, 8, BASE, 8, FREE)[0] == -1
    assert m.i8_scaled_path("k_contig", 8, 8, 0, BASE, 1, BASE, 1, FREE)[0] == TINY
    assert m.i8_scaled_path("k_contig", 1, 64, 64, BASE, 64, BASE, 64, 0) == (STREAM, {"panel": 0, "ranges": 1, "streamk_tiles": 0, "workspace": 0})
    assert m.grad_i8_path("f32", "k_contig", 8, 8, 8, BASE, 8, BASE, 8, "f32", FREE)[0] == -1
    assert m.grad_i8_path("bf16", "k_contig", 8, 8, -1, BASE, 8, BASE, 8, "f32", FREE)[0] == -1
    assert m.grad_i8_path("bf16", "k_contig", 1, 1, 1, BASE, 1, BASE, 1, "f32", FREE)[0] == TINY
    assert m.grad_i8_path("bf16", "k_contig", 1, 1000, 500, BASE, 500, BASE, 1000, "bf16", 0)[0] == GENERAL


@pytest.mark.parametrize("case", cases.SCALED, ids=str)
def test_scaled_cases_plan_the_forms_they_are_for(case):
    layout, M, N, K, aligned, ws, kernel, panels, streamk, ranges = case
    lda, ldb = cases.scaled_lds(layout, M, N, K, aligned)
    got, p = m.i8_scaled_path(layout, M, N, K, BASE, lda, BASE, ldb, ws)
    assert (got, -(-N // p["panel"]) if p["panel"] else 0, p["streamk_tiles"], p["ranges"]) == (kernel, panels, streamk, ranges), p
    assert panels < 2 or N % p["panel"]  # a last panel of its own width


@pytest.mark.parametrize("dtA", ["bf16", "f16"])
@pytest.mark.parametrize("case", cases.GRAD, ids=str)
def test_gradient_cases_plan_the_forms_they_are_for(case, dtA):
    dtD, layout, M, N, K, aligned, ws, kernel, panels, streamk = case
    got, p = m.grad_i8_path(dtA, layout, M, N, K, BASE, cases.grad_lda(layout, M, K, aligned), BASE, N, "f32" if dtD == "f32" else dtA, ws)
    assert (got, -(-N // p["panel"]) if p["panel"] else 0, p["streamk_tiles"]) == (kernel, panels, streamk), p
    assert panels < 2 or N % p["panel"]


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_the_bound_for_few_nonzeros_tells_a_missing_rest(dt):
    # the kernels' two values in binary64: within the bound; without the rest far outside
    M, N, K, n = 40, 60, 4096, 4
    a = cases.few_nonzeros(1, M, K, n, dt)
    q, s = cases.grad_inputs(2, K, N)
    d, mag = ref.grad_i8(a, q, s, None, 0.0)
    tol = cases.sparse_grad_tol(dt, a, d, mag, n)
    hi, lo = cases.split_values(q, s, dt)
    A = a.double()
    assert bool(((A @ (hi + lo) - d).abs() <= tol).all())
    bad = (A @ hi - d).abs() / tol
    assert float(bad.max()) > 20 and float((bad > 1).double().mean()) > 0.9, bad.max()
    for wrong in (A @ (hi - lo), A @ (hi + lo.roll(1, 1)), A @ (hi + lo.roll(1, 0))):  # a sign, a column or a row off
        assert float((wrong - d).abs().div(tol).max()) > 20
