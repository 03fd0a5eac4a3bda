"""GPU parity of the 8-bit linear layer with its plain binary64 forms: every type,
odd and strided rows, single tokens, empty and non-finite rows, aliases, K ranges
and streams.  Tolerances count roundings (linear8_ref.U, half a step each)."""
import numpy as np
import pytest
import torch

import linear8_ref as ref
from gpu_util import need_gpu, say
from linear8_ref import DT, SUB, U, U32

pytestmark = pytest.mark.gpu
GUARD = -77  # what strided() puts around int8 rows


def put(t, pad=0, offset=0):
    """A device copy of t in a strided buffer."""
    v = ref.strided(t.shape[0], t.shape[1], pad, t.dtype, "cuda", offset)
    v.copy_(t)
    return v


def empty(rows, cols, dtype, pad=0, offset=0):
    return ref.strided(rows, cols, pad, dtype, "cuda", offset)


def ld(t):
    return 0 if t is None else t.stride(0)


def guards_hold(*views):
    torch.cuda.synchronize()
    for v in views:
        if v is None or v.stride(0) == v.shape[1]:
            continue
        rest = v.as_strided((v.shape[0], v.stride(0)), v.stride())[:, v.shape[1]:]
        assert bool((rest == GUARD).all() if v.dtype == torch.int8 else torch.isnan(rest).all()), "wrote between the rows"


def within(got, exact, tol, what):
    d = (got.double().cpu() - exact).abs()
    bad = ~(d <= tol)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {float((d / tol).nan_to_num(1e30).max())} of the tolerance"


# --------------------------------------------------------------------- norm
NORM_SHAPES = [(1, 1), (1, 8), (3, 7), (5, 64), (2, 511), (4, 513), (9, 1000), (3, 1025), (2, 2048), (7, 2051), (3, 4096),
               (2, 5000), (300, 5120), (1, 8192), (2, 8200), (2, 16384), (2, 16390), (1, 40000), (1000, 96)]


def check_codes(q, scale, y, what):
    """Codes against exact rows y: the scale is one binary32 value off by the row's
    statistics (under 2^-16 for rows of up to 2^16: 64 sums of 2^-24 along the
    longest chain and a square root), a code by half a step and by 127 times the
    rounding of y / scale (8 roundings)."""
    top = y.abs().amax(1)
    within(scale, top / 127, 2.0 ** -16 * top / 127 + 1e-44, what + " scale")
    s = (top / 127)[:, None]
    d = (q.double().cpu() * s - y).abs()
    assert bool((d <= s * (0.5 + 127 * 8 * U32)).all()), what + " codes"
    assert int(q.abs().max()) <= 127


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", NORM_SHAPES, ids=str)
def test_rmsnorm_quant(dt, shape):
    mcg = need_gpu()
    M, N = shape
    seed = M * 131 + N
    for residual, weight, pad, off in ((True, True, 0, 0), (False, False, 3, 1)):
        x = ref.rand(seed, M, N, gain=2).to(DT[dt])
        r = ref.rand(seed + 1, M, N).to(DT[dt]) if residual else None
        w = (1 + 0.3 * ref.rand(seed + 2, N)).to(DT[dt]) if weight else None
        dx, dr = put(x, pad, off), None if r is None else put(r, pad + 1, off)
        H, Q = empty(M, N, DT[dt], pad, off), empty(M, N, torch.int8, pad, off)
        scale, rstd = torch.full((M,), float("nan"), device="cuda"), torch.full((M,), float("nan"), device="cuda")
        mcg.rmsnorm_quant(dt, M, N, dx, ld(dx), dr, ld(dr), None if w is None else w.cuda(), 1e-5, H, ld(H), Q, ld(Q),
                          scale, rstd)
        guards_hold(H, Q)
        h, y, rs = ref.rmsnorm(x, r, w, 1e-5)
        within(H, h, (U[dt] + U32) * h.abs() + SUB[dt], "h")
        within(rstd, rs, 2.0 ** -17 * rs, "rstd")
        check_codes(Q, scale, y, f"{dt} {shape}")


def test_rmsnorm_quant_in_place_and_without_outputs():
    mcg = need_gpu()
    for N in (777, 20000):  # a row in registers, and a row read twice
        x, r = ref.rand(1, 5, N).to(torch.bfloat16), ref.rand(2, 5, N).to(torch.bfloat16)
        outs = []
        for target in ("new", "x", "r", "none"):
            dx, dr = put(x), put(r)
            H = {"new": empty(5, N, torch.bfloat16), "x": dx, "r": dr, "none": None}[target]
            Q, scale = empty(5, N, torch.int8), torch.empty(5, device="cuda")
            mcg.rmsnorm_quant("bf16", 5, N, dx, N, dr, N, None, 1e-6, H, N, Q, N, scale)
            torch.cuda.synchronize()
            outs.append((None if H is None else H.clone(), Q, scale))
            if target != "x":
                assert torch.equal(dx.cpu(), x)
            if target != "r":
                assert torch.equal(dr.cpu(), r)
        for H, Q, scale in outs[1:]:
            assert H is None or torch.equal(H, outs[0][0])
            assert torch.equal(Q, outs[0][1]) and torch.equal(scale, outs[0][2])


@pytest.mark.parametrize("N", [5, 300, 3000, 20000])
def test_rows_that_hold_nothing_or_no_number(N):
    mcg = need_gpu()
    M = 9
    x = ref.rand(5, M, N).float()
    x[0] = 0
    x[1, N // 2] = float("nan")
    x[2, 0] = float("inf")
    x[3, N - 1] = float("-inf")
    x[4] = x[4] * 1e-42  # subnormal rows
    x[5] = x[5] * 1e-36
    x[6] = x[6] * 1e30   # squares leave binary32
    x[7] = -0.0
    X = put(x)
    Q, scale, rstd = empty(M, N, torch.int8), torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    mcg.rmsnorm_quant("f32", M, N, X, N, None, 0, None, 1e-5, None, 0, Q, N, scale, rstd)
    torch.cuda.synchronize()
    q, s = Q.cpu(), scale.cpu()
    assert not q[[0, 1, 2, 3, 6, 7]].any() and s[0] == 0 and s[7] == 0
    assert bool(torch.isnan(s[[1, 2, 3, 6]]).all())
    for i in (4, 5):  # tiny rows keep their shape: codes reach the end of the range
        assert int(q[i].abs().max()) == 127
    check_codes(Q[8:], scale[8:], ref.rmsnorm(x[8:], None, None, 1e-5)[1], "a row beside them")
    # eps 0: the zero row has an infinite rstd and still the scale 0
    mcg.rmsnorm_quant("f32", M, N, X, N, None, 0, None, 0.0, None, 0, Q, N, scale, rstd)
    torch.cuda.synchronize()
    assert float(scale[0]) == 0 and not Q[0].any()
    # the same rows without the norm: large finite rows are rows like any other
    mcg.quantize_rows("f32", M, N, X, N, Q, N, scale)
    D = empty(M, N, torch.float32)
    mcg.dequantize_rows("f32", M, N, Q, N, scale, D, N)
    torch.cuda.synchronize()
    s = scale.cpu()
    assert s[0] == 0 and bool(torch.isnan(s[[1, 2, 3]]).all()) and not Q[[0, 1, 2, 3, 7]].any()
    assert bool(torch.isnan(D[[1, 2, 3]]).all()) and not D[[0, 7]].any()
    for i in (5, 6, 8):
        check_codes(Q[i:i + 1], scale[i:i + 1], x[i:i + 1].double(), f"row {i}")
    assert int(Q[4].abs().max()) == 127


def test_rows_of_length_zero():
    mcg = need_gpu()
    scale, rstd = torch.full((3,), 7.0, device="cuda"), torch.full((3,), 7.0, device="cuda")
    mcg.rmsnorm_quant("bf16", 3, 0, None, 1, None, 0, None, 0.25, None, 0, None, 1, scale, rstd)
    torch.cuda.synchronize()
    assert scale.cpu().tolist() == [0, 0, 0] and rstd.cpu().tolist() == [2, 2, 2]
    scale.fill_(7)
    mcg.quantize_rows("f16", 3, 0, None, 1, None, 1, scale)
    torch.cuda.synchronize()
    assert scale.cpu().tolist() == [0, 0, 0]


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", [(1, 1), (1, 8), (3, 7), (70, 130), (2, 1030), (33, 2049), (5, 8192), (2, 9000), (1, 33000)], ids=str)
def test_quantize_and_dequantize_rows(dt, shape):
    mcg = need_gpu()
    M, N = shape
    for pad, off in ((0, 0), (5, 3)):
        x = ref.rand(M + N, M, N, gain=3).to(DT[dt])
        X, Q, scale = put(x, pad, off), empty(M, N, torch.int8, pad, off), torch.empty(M, device="cuda")
        mcg.quantize_rows(dt, M, N, X, ld(X), Q, ld(Q), scale)
        check_codes(Q, scale, x.double(), f"{dt} {shape}")
        for do in DT:
            D = empty(M, N, DT[do], pad, off)
            mcg.dequantize_rows(do, M, N, Q, ld(Q), scale, D, ld(D))
            guards_hold(Q, D)
            v = Q.cpu().double() * scale.cpu().double()[:, None]
            within(D, v, (U[do] + U32) * v.abs() + SUB[do], f"values in {do}")


# ----------------------------------------------------------------- gradient
def run_backward(mcg, dt, M, N, dy, x, scale, w, rstd, dr, pad=0, off=0, want_dw=True, into=None):
    DY, X = put(dy, pad, off), put(x, pad, off)
    DR = None if dr is None else put(dr, pad + 2, off)
    DX = {None: None, "dy": DY, "dr": DR}[into]
    DX = empty(M, N, DT[dt], pad, off) if DX is None else DX
    DW = torch.full((N,), float("nan"), device="cuda") if want_dw else None
    ws = torch.full((max(1, mcg.rmsnorm_backward_workspace_bytes(M, N)) // 4 + 4,), float("nan"), device="cuda")
    mcg.rmsnorm_backward(dt, "i8" if scale is not None else dt, M, N, DY, ld(DY), X, ld(X), None if scale is None else scale.cuda(),
                         None if w is None else w.cuda(), rstd.cuda(), DR, ld(DR), DX, ld(DX), DW, ws if want_dw else None)
    guards_hold(DX)
    return DX, DW


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("x8", [False, True], ids=["x", "x8"])
@pytest.mark.parametrize("shape", [(1, 1), (1, 64), (5, 7), (600, 70), (2, 513), (40, 1000), (3, 2048), (1300, 2050), (4, 4099), (6, 8192),
                                   (3, 9001), (2, 16384), (3, 16385), (2, 40000)], ids=str)
def test_rmsnorm_backward(dt, x8, shape):
    mcg = need_gpu()
    M, N = shape
    for full, pad, off in ((True, 0, 0), (False, 5, 1)):
        dy = ref.rand(N, M, N).to(DT[dt])
        w = (1 + 0.3 * ref.rand(N + 2, N)).to(DT[dt]) if full else None
        dr = ref.rand(N + 3, M, N).to(DT[dt]) if full else None
        if x8:
            x, scale = ref.codes(N + 1, M, N), ref.rand(N + 4, M).abs().float() * 0.02 + 1e-3
            xv = x.double() * scale.double()[:, None]
        else:
            x, scale = ref.rand(N + 1, M, N, gain=2).to(DT[dt]), None
            xv = x.double()
        rstd = ref.rmsnorm(xv, None, None, 1e-5)[2].float()
        DX, DW = run_backward(mcg, dt, M, N, dy, x, scale, w, rstd, dr, pad, off)
        dx, dw = ref.rmsnorm_backward(dy, xv, w, rstd, dr)
        # dx = rstd (g - c x) + dr: c's sum of N products is off by at most (L + 3) u of
        # the products' magnitudes, L the longest chain (16 per thread or N / 1024 in the
        # long rows, 6 in the wavefront, 16 over wavefronts); each term a few roundings
        g = dy.double() if w is None else dy.double() * w.double()
        r = rstd.double()[:, None]
        L = 64 + N // 1024
        c = r.square() * (g * xv).abs().mean(1, keepdim=True)
        terms = r * (g.abs() + c * xv.abs()) + (0 if dr is None else dr.double().abs())
        within(DX, dx, L * U32 * terms + U[dt] * dx.abs() + SUB[dt], f"dx {dt} {shape}")
        # dw: a chain of at most M / parts rows, then parts / 8 and 8 partial rows
        mag = (dy.double() * xv * r).abs().sum(0)
        within(DW, dw, (M // 512 + 160) * U32 * mag + 1e-45, f"dw {dt} {shape}")


def test_rmsnorm_backward_in_place_without_dw_and_empty():
    mcg = need_gpu()
    for N in (1000, 20000):
        M = 7
        dy, x, dr = (ref.rand(i, M, N).to(torch.bfloat16) for i in (1, 2, 3))
        rstd = ref.rmsnorm(x, None, None, 1e-5)[2].float()
        base, dw = run_backward(mcg, "bf16", M, N, dy, x, None, None, rstd, dr)
        for into in ("dy", "dr"):
            got, dw2 = run_backward(mcg, "bf16", M, N, dy, x, None, None, rstd, dr, into=into)
            assert torch.equal(got.contiguous(), base.contiguous()) and torch.equal(dw, dw2), into
        got, none = run_backward(mcg, "bf16", M, N, dy, x, None, None, rstd, dr, want_dw=False)
        assert none is None and torch.equal(got, base)
    dw = torch.full((33,), 5.0, device="cuda")
    mcg.rmsnorm_backward("f32", "f32", 0, 33, None, 1, None, 1, None, None, None, None, 0, None, 1, dw)
    torch.cuda.synchronize()
    assert not dw.any()


def test_rmsnorm_backward_against_differences():
    # the binary32 kernels against central differences of the plain forward pass in binary64
    mcg = need_gpu()
    M, N, eps, e = 2, 130, 1e-5, 1e-5
    x, w, dy = ref.rand(1, M, N).float(), (1 + 0.3 * ref.rand(2, N)).float(), ref.rand(3, M, N).float()
    rstd = ref.rmsnorm(x, None, w, eps)[2].float()
    DX, DW = run_backward(mcg, "f32", M, N, dy, x, None, w, rstd, None)

    def loss(x, w):
        return float((ref.rmsnorm(x, None, w, eps)[1] * dy.double()).sum())
    # differences: 1e-8 (see test_linear8_ref); the kernel: 64 u of terms of order 10
    for j in range(0, N, 7):
        for i in range(M):
            d = torch.zeros(M, N, dtype=torch.float64)
            d[i, j] = e
            assert abs((loss(x.double() + d, w) - loss(x.double() - d, w)) / (2 * e) - float(DX[i, j])) < 1e-8 + 64 * U32 * 10
        d = torch.zeros(N, dtype=torch.float64)
        d[j] = e
        assert abs((loss(x, w.double() + d) - loss(x, w.double() - d)) / (2 * e) - float(DW[j])) < 1e-8 + 64 * U32 * 10


# ----------------------------------------------------------------- products
SCALED_SHAPES = [(1, 1, 1), (1, 64, 64), (1, 1000, 4096), (3, 17, 5), (7, 130, 257), (16, 256, 1024), (31, 100, 2000), (32, 4096, 512),
                 (33, 129, 127), (100, 300, 4100), (128, 128, 16384), (129, 257, 1000), (256, 256, 256), (300, 520, 640),
                 (513, 384, 1024), (640, 768, 4096), (1, 5000, 16400), (2, 300, 40000)]


def run_scaled(mcg, a, sa, b, sb, bias, dt, layoutB, pads=(0, 0, 0), off=0, ws=None, d=None):
    """a M x K, b K x N on the CPU; returns D."""
    M, K = a.shape
    N = b.shape[1]
    A = put(a, pads[0], off)
    B = put(b.T.contiguous() if layoutB == "k_contig" else b, pads[1], off)
    D = empty(M, N, DT[dt], pads[2], off) if d is None else d
    mcg.gemm_i8_scaled(layoutB, M, N, K, A, ld(A), sa.cuda(), B, ld(B), sb.cuda(), None if bias is None else bias.cuda(),
                       D, ld(D), dt, ws)
    guards_hold(D)
    return D


def scaled_tol(d, core, bias, dt):
    """binary32 of the sum, times sa, times sb with the bias: three roundings of the
    product and one of the result, then D's."""
    return 3 * U32 * core.abs() + U32 * d.abs() + (U[dt] if dt != "f32" else 0) * d.abs() * (1 + 1e-6) + SUB[dt]


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("layoutB", ["k_contig", "mn_contig"])
@pytest.mark.parametrize("shape", SCALED_SHAPES, ids=str)
def test_gemm_i8_scaled(dt, layoutB, shape):
    mcg = need_gpu()
    M, N, K = shape
    a, b = ref.codes(K, M, K), ref.codes(K + 1, K, N)
    sa, sb = ref.rand(M, M).abs().float() * 0.01 + 1e-3, ref.rand(N, N).abs().float() * 1e-3 + 1e-4
    for bias, pads, off, ws in ((None, (0, 0, 0), 0, None), (ref.rand(3, N).float(), (0, 0, 0), 0, 32 << 20),
                                (None, (16, 32, 4), 0, 3 * M * N * 4), (ref.rand(4, N).float(), (1, 3, 5), 1, 32 << 20)):
        w = None if ws is None else torch.full((ws // 4 + 4,), 0x7B7B7B7B, dtype=torch.int32, device="cuda")
        D = run_scaled(mcg, a, sa, b, sb, bias, dt, layoutB, pads, off, w)
        core = ref.i8_scaled(a, sa, b, sb, None)
        d = core if bias is None else core + bias.double()
        within(D, d, scaled_tol(d, core, bias, dt), f"{dt} {layoutB} {shape} pads {pads}")


def test_gemm_i8_scaled_extremes():
    mcg = need_gpu()
    # the largest sums, at the largest K: exact int32, no wrap
    K = 131071
    a, b = torch.full((2, K), -128, dtype=torch.int8), torch.full((K, 3), -128, dtype=torch.int8)
    one = torch.ones(3)
    D = run_scaled(mcg, a, one[:2], b, one, None, "f32", "k_contig")
    assert D.cpu().tolist() == [[float(np.float32(16384.0 * K))] * 3] * 2
    # K = 0: the bias alone
    bias = torch.tensor([1.0, -2.0, 3.0])
    D = empty(2, 3, torch.float32)
    mcg.gemm_i8_scaled("k_contig", 2, 3, 0, None, 1, one.cuda(), None, 1, one.cuda(), bias.cuda(), D, 3, "f32")
    torch.cuda.synchronize()
    assert D.cpu().tolist() == [bias.tolist()] * 2
    # a scale that is no number marks its row or column and nothing else
    a, b = ref.codes(1, 40, 300), ref.codes(2, 300, 50)
    sa, sb = torch.ones(40), torch.ones(50)
    sa[7], sb[11] = float("nan"), float("inf")
    D = run_scaled(mcg, a, sa, b, sb, None, "bf16", "k_contig").cpu()
    assert bool(torch.isnan(D[7]).all()) and not bool(torch.isfinite(D[:, 11]).any())
    D[7], D[:, 11] = 0, 0
    assert bool(torch.isfinite(D).all())


def test_gemm_i8_scaled_result_does_not_depend_on_the_workspace():
    mcg = need_gpu()
    for M, N, K in ((5, 700, 4096), (130, 260, 8192), (64, 512, 6000)):
        a, b = ref.codes(1, M, K), ref.codes(2, K, N)
        sa, sb = ref.rand(3, M).abs().float(), ref.rand(4, N).abs().float()
        base = run_scaled(mcg, a, sa, b, sb, None, "f32", "k_contig")
        need = mcg.i8_scaled_workspace_bytes("k_contig", M, N, K, None, K, None, K)
        for nb in (16, need // 2, need, need + 4096):
            ws = torch.empty(max(1, nb), dtype=torch.uint8, device="cuda")
            assert torch.equal(run_scaled(mcg, a, sa, b, sb, None, "f32", "k_contig", ws=ws), base), (M, N, K, nb)


@pytest.mark.parametrize("layoutB", ["k_contig", "mn_contig"])
@pytest.mark.parametrize("shape", [(600, 1300, 2050), (1300, 700, 1999), (1001, 2003, 3001)], ids=str)
def test_gemm_i8_scaled_unaligned_operands_in_panels(layoutB, shape):
    # operands without 16-byte chunks on the copies in the workspace, whole and in panels:
    # the sums are exact, so every way gives the same bits
    mcg = need_gpu()
    M, N, K = shape
    a, b = ref.codes(1, M, K), ref.codes(2, K, N)
    sa, sb = ref.rand(3, M).abs().float() + 0.1, ref.rand(4, N).abs().float() + 0.1
    bias = ref.rand(5, N).float()
    pads = (5, 7, 3)
    base = run_scaled(mcg, a, sa, b, sb, bias, "f32", layoutB, pads, 1)
    d = ref.i8_scaled(a, sa, b, sb, bias)
    within(base, d, scaled_tol(d, d - bias.double(), bias, "f32"), f"{layoutB} {shape}")
    copy = (M + 512) * (K + 16) + 4096
    for nb in (copy, copy + 300 * (K + 16), 64 << 20):
        ws = torch.full((nb,), 0x7B, dtype=torch.uint8, device="cuda")
        assert torch.equal(run_scaled(mcg, a, sa, b, sb, bias, "f32", layoutB, pads, 1, ws), base), nb


GRAD_SHAPES = [(1, 1, 1), (3, 5, 7), (64, 64, 64), (100, 130, 257), (128, 128, 4096), (129, 255, 1000), (256, 512, 333), (300, 300, 2),
               (256, 256, 2048), (512, 384, 640), (520, 776, 1032), (1, 1000, 500), (1000, 1, 300)]


@pytest.mark.parametrize("dtA", ["bf16", "f16"])
@pytest.mark.parametrize("layoutA", ["k_contig", "mn_contig"])
@pytest.mark.parametrize("shape", GRAD_SHAPES, ids=str)
def test_gemm_grad_i8(dtA, layoutA, shape):
    mcg = need_gpu()
    M, N, K = shape
    a = ref.rand(K, M, K).to(DT[dtA])
    q, s = ref.codes(K + 1, K, N), ref.rand(K + 2, K).abs().float() * 0.02 + 1e-3
    for dtD, beta, pads, off, ws in ((dtA, 0.0, (0, 0, 0), 0, None), ("f32", 1.0, (0, 0, 0), 0, 32 << 20), (dtA, -0.5, (8, 16, 4), 0, 32 << 20),
                                     ("f32", 0.0, (3, 1, 5), 1, 3 * M * N * 4), (dtA, 1.0, (1, 7, 3), 1, 32 << 20)):
        A = put(a if layoutA == "k_contig" else a.T.contiguous(), pads[0], off)
        Q = put(q, pads[1], off)
        c = ref.rand(K + 3, M, N).to(DT[dtD]) if beta else None
        C = None if c is None else put(c, pads[2], off)
        D = empty(M, N, DT[dtD], pads[2], off)
        w = None if ws is None else torch.full((ws // 4 + 4,), float("nan"), device="cuda")
        mcg.gemm_grad_i8(dtA, layoutA, M, N, K, A, ld(A), Q, ld(Q), s.cuda(), C, D, ld(D), dtD, beta, w)
        guards_hold(D)
        d, mag = ref.grad_i8(a, q, s, c, beta)
        # a product's 8-bit side: formed with one binary32 rounding, then rounded to A's
        # type (or the rest of two roundings left: U^2, and the spacing near zero); the
        # matrix cores' sum 4 u (K + 2); C's step and D's
        operand = U[dtA] if dtD != "f32" else U[dtA] ** 2
        near0 = SUB[dtA] * (a.double().abs().sum(1, keepdim=True))
        tol = (operand + (4 * (K + 2) + 1) * U32) * mag + near0 + 2 * U32 * d.abs() + (0 if c is None else U32 * abs(beta) * c.double().abs())
        if dtD != "f32":
            tol = tol + U[dtD] * (d.abs() + tol) + SUB[dtD]
        within(D, d, tol, f"{dtA} -> {dtD} {layoutA} {shape} pads {pads}")
        if c is not None:  # D may be C
            mcg.gemm_grad_i8(dtA, layoutA, M, N, K, A, ld(A), Q, ld(Q), s.cuda(), C, C, ld(C), dtD, beta, w)
            torch.cuda.synchronize()
            assert torch.equal(C, D)


def grad_tol(dtA, dtD, a, s, d, mag, K):
    """As in test_gemm_grad_i8, with one more binary32 rounding for a result added up
    from two products."""
    operand = U[dtA] if dtD != "f32" else U[dtA] ** 2
    near0 = SUB[dtA] * (a.double().abs().sum(1, keepdim=True))
    tol = (operand + (4 * (K + 2) + 1) * U32) * mag + near0 + 4 * U32 * d.abs()
    return tol if dtD == "f32" else tol + U[dtD] * (d.abs() + tol) + SUB[dtD]


@pytest.mark.parametrize("dtA", ["bf16", "f16"])
@pytest.mark.parametrize("layoutA", ["k_contig", "mn_contig"])
@pytest.mark.parametrize("shape", [(512, 1536, 4096), (600, 900, 700), (1001, 1103, 901)], ids=str)
def test_gemm_grad_i8_in_panels(dtA, layoutA, shape):
    # panels of the widened Q in the workspace: whole, cut along N, and with a copy of an A
    # without 16-byte chunks
    mcg = need_gpu()
    M, N, K = shape
    a = ref.rand(K, M, K).to(DT[dtA])
    q, s = ref.codes(K + 1, K, N), ref.rand(K + 2, K).abs().float() * 0.02 + 1e-3
    core, mag = ref.grad_i8(a, q, s, None, 0.0)
    c = ref.rand(K + 3, M, N)
    for dtD, beta, pad in ((dtA, 0.0, 0), ("f32", 1.0, 0), ("f32", 0.0, 3), (dtA, -0.5, 5)):
        A = put(a if layoutA == "k_contig" else a.T.contiguous(), pad)
        Q = put(q, pad)
        C = put(c.to(DT[dtD]), pad)
        d = core + beta * c.to(DT[dtD]).double() if beta else core
        full = mag + (abs(beta) * c.abs() if beta else 0)
        two = 2 if dtD == "f32" else 1
        copy = (M + 8) * (K + 8) * 2
        for nb in (copy + 600 * (K + 8) * 2 * two, 64 << 20):
            ws = torch.full((nb // 4,), float("nan"), device="cuda")
            D = empty(M, N, DT[dtD], pad)
            mcg.gemm_grad_i8(dtA, layoutA, M, N, K, A, ld(A), Q, ld(Q), s.cuda(), C if beta else None, D, ld(D), dtD, beta, ws)
            guards_hold(D)
            within(D, d, grad_tol(dtA, dtD, a, s, d, full, K), f"{dtA} -> {dtD} {layoutA} {shape} beta {beta} workspace {nb}")


def test_gemm_grad_i8_empty_sum_and_marked_rows():
    mcg = need_gpu()
    C = put(ref.rand(1, 3, 5).float())
    D = empty(3, 5, torch.float32)
    mcg.gemm_grad_i8("bf16", "k_contig", 3, 5, 0, None, 1, None, 5, None, C, D, 5, "f32", 2.0)
    torch.cuda.synchronize()
    assert torch.equal(D, 2 * C)
    # a row whose scale is NaN (it held no number when it was put in 8 bits) shows in every output
    a, q, s = ref.rand(1, 20, 70).to(torch.bfloat16), ref.codes(2, 70, 30), torch.ones(70)
    s[69] = float("nan")
    D = empty(20, 30, torch.bfloat16)
    mcg.gemm_grad_i8("bf16", "k_contig", 20, 30, 70, put(a), 70, put(q), 30, s.cuda(), None, D, 30, "bf16")
    torch.cuda.synchronize()
    assert bool(torch.isnan(D).all())
    # the sum ends at K: rows past it are not read
    mcg.gemm_grad_i8("bf16", "k_contig", 20, 30, 69, put(a), 70, put(q), 30, s.cuda(), None, D, 30, "bf16")
    torch.cuda.synchronize()
    assert bool(torch.isfinite(D).all())


@pytest.mark.parametrize("layoutB", ["k_contig", "mn_contig"])
@pytest.mark.parametrize("shape", [(100, 70, 5), (40, 3, 9), (3, 300, 15), (17, 15, 300), (2, 7, 1), (5, 3, 40)], ids=str)
def test_gemm_i8_scaled_rows_shorter_than_a_chunk(layoutB, shape):
    # rows of fewer than 16 bytes, and whole operands of fewer
    mcg = need_gpu()
    M, N, K = shape
    a, b = ref.codes(K, M, K), ref.codes(K + 1, K, N)
    sa, sb, bias = ref.rand(1, M).abs().float() + 0.1, ref.rand(2, N).abs().float() + 0.1, ref.rand(3, N).float()
    d = ref.i8_scaled(a, sa, b, sb, bias)
    for pads, off in (((0, 0, 0), 0), ((1, 2, 3), 1), ((16, 16, 4), 0)):
        D = run_scaled(mcg, a, sa, b, sb, bias, "f32", layoutB, pads, off, torch.empty(1 << 20, dtype=torch.uint8, device="cuda"))
        within(D, d, scaled_tol(d, d - bias.double(), bias, "f32"), f"{layoutB} {shape} pads {pads}")


@pytest.mark.parametrize("layoutA", ["k_contig", "mn_contig"])
@pytest.mark.parametrize("shape", [(3, 200, 40), (100, 70, 5), (2, 300, 500), (5, 130, 3), (1, 15, 1), (7, 2, 1), (33, 9, 70), (1, 3, 200)], ids=str)
def test_gemm_grad_i8_rows_shorter_than_a_chunk(layoutA, shape):
    mcg = need_gpu()
    M, N, K = shape
    a = ref.rand(K, M, K).to(torch.bfloat16)
    q, s = ref.codes(K + 1, K, N), ref.rand(K + 2, K).abs().float() * 0.02 + 1e-3
    c = ref.rand(K + 3, M, N)
    for dtD, beta, pad, off in (("bf16", 0.0, 0, 0), ("f32", -0.5, 3, 1), ("bf16", 1.0, 16, 0)):
        A, Q, C = put(a if layoutA == "k_contig" else a.T.contiguous(), pad, off), put(q, pad, off), put(c.to(DT[dtD]), pad, off)
        d, mag = ref.grad_i8(a, q, s, c.to(DT[dtD]) if beta else None, beta)
        if beta:
            mag = mag + abs(beta) * c.abs()
        D = empty(M, N, DT[dtD], pad, off)
        mcg.gemm_grad_i8("bf16", layoutA, M, N, K, A, ld(A), Q, ld(Q), s.cuda(), C if beta else None, D, ld(D), dtD, beta,
                         torch.empty(1 << 20, dtype=torch.uint8, device="cuda"))
        guards_hold(D)
        within(D, d, grad_tol("bf16", dtD, a, s, d, mag, K), f"{layoutA} {shape} -> {dtD} beta {beta} pad {pad}")


# Products on the 256 x 256 and stream-K forms, by sampled rows: first and last, and a
# few of every tile.
def sampled(M):
    return sorted({0, 1, M - 1, M - 2, *range(5, M, 97)})


@pytest.mark.parametrize("layoutB", ["k_contig", "mn_contig"])
@pytest.mark.parametrize("shape", [(4352, 4352, 1024), (4217, 4100, 560), (8192, 1040, 2064)], ids=str)
def test_large_scaled_products_by_sampled_rows(layoutB, shape):
    mcg = need_gpu()
    M, N, K = shape
    a, b = ref.codes(1, M, K), ref.codes(2, K, N)
    sa, sb, bias = ref.rand(3, M).abs().float() + 0.1, ref.rand(4, N).abs().float() + 0.1, ref.rand(5, N).float()
    rows = sampled(M)
    d = ref.i8_scaled(a[rows], sa[rows], b, sb, bias)
    core = d - bias.double()
    for dt, ws in (("bf16", None), ("f32", 64 << 20)):
        w = None if ws is None else torch.full((ws,), 0x7B, dtype=torch.uint8, device="cuda")
        D = run_scaled(mcg, a, sa, b, sb, bias, dt, layoutB, ws=w)
        within(D[rows], d, scaled_tol(d, core, bias, dt), f"{dt} {layoutB} {shape}")


@pytest.mark.parametrize("layoutA", ["k_contig", "mn_contig"])
@pytest.mark.parametrize("shape", [(4352, 4352, 520), (4217, 4100, 1033), (4090, 4090, 1033)], ids=str)
def test_large_gradient_products_by_sampled_rows(layoutA, shape):
    mcg = need_gpu()
    M, N, K = shape
    a = ref.rand(1, M, K).to(torch.bfloat16)
    q, s = ref.codes(2, K, N), ref.rand(3, K).abs().float() * 0.02 + 1e-3
    rows = sampled(M)
    d, mag = ref.grad_i8(a[rows], q, s, None, 0.0)
    for dtD, ws in (("bf16", 64 << 20), ("f32", 64 << 20), ("bf16", 14 << 20)):
        A, Q = put(a if layoutA == "k_contig" else a.T.contiguous()), put(q)
        D = empty(M, N, DT[dtD])
        w = torch.full((ws // 4,), float("nan"), device="cuda")
        mcg.gemm_grad_i8("bf16", layoutA, M, N, K, A, ld(A), Q, ld(Q), s.cuda(), None, D, ld(D), dtD, 0.0, w)
        torch.cuda.synchronize()
        assert bool(torch.isfinite(D).all())
        within(D[rows], d, grad_tol("bf16", dtD, a[rows], s, d, mag, K), f"{dtD} {layoutA} {shape} workspace {ws}")


# ------------------------------------------------------------ a layer's step
def layer_step(mcg, s, T, K, N, stream=None):
    """Forward and backward of norm + linear in 8 bits on the buffers of s."""
    mcg.rmsnorm_quant("bf16", T, K, s["x"], K, s["r"], K, s["w"], 1e-5, s["h"], K, s["q"], K, s["sx"], s["rstd"], stream)
    mcg.gemm_i8_scaled("k_contig", T, N, K, s["q"], K, s["sx"], s["qw"], K, s["sw"], None, s["y"], N, "bf16", s["ws"], stream=stream)
    mcg.gemm_grad_i8("bf16", "k_contig", T, K, N, s["dy"], N, s["qw"], K, s["sw"], None, s["dx"], K, "bf16", 0.0, s["ws"], stream=stream)
    mcg.gemm_grad_i8("bf16", "mn_contig", N, K, T, s["dy"], N, s["q"], K, s["sx"], None, s["dw"], K, "f32", 0.0, s["ws"], stream=stream)
    mcg.rmsnorm_backward("bf16", "bf16", T, K, s["dx"], K, s["h"], K, None, s["w"], s["rstd"], None, 0, s["dh"], K, s["dg"], s["ws"], stream=stream)


def layer_state(T, K, N):
    c = lambda t: t.cuda()
    bf = torch.bfloat16
    qw = ref.codes(9, N, K)
    return {"x": c(ref.rand(1, T, K).to(bf)), "r": c(ref.rand(2, T, K).to(bf)), "w": c((1 + 0.1 * ref.rand(3, K)).to(bf)),
            "h": empty(T, K, bf), "q": empty(T, K, torch.int8), "sx": torch.empty(T, device="cuda"), "rstd": torch.empty(T, device="cuda"),
            "qw": c(qw), "sw": c((ref.rand(4, N).abs() * 1e-3 + 1e-4).float()), "y": empty(T, N, bf), "dy": c(ref.rand(5, T, N).to(bf)),
            "dx": empty(T, K, bf), "dw": empty(N, K, torch.float32), "dh": empty(T, K, bf), "dg": torch.empty(K, device="cuda"),
            "ws": torch.empty(32 << 20, dtype=torch.uint8, device="cuda")}


OUTS = ("h", "q", "sx", "rstd", "y", "dx", "dw", "dh", "dg")


@pytest.mark.parametrize("shape", [(1, 512, 256), (37, 500, 333), (300, 1024, 768)], ids=str)
def test_a_layers_step_on_another_stream_and_in_a_graph(shape):
    mcg = need_gpu()
    T, K, N = shape
    s = layer_state(T, K, N)
    layer_step(mcg, s, T, K, N)
    torch.cuda.synchronize()
    eager = {k: s[k].clone() for k in OUTS}

    def reset():
        for k in OUTS:
            s[k].fill_(-77 if s[k].dtype == torch.int8 else float("nan"))
        torch.cuda.synchronize()

    def same(what):
        torch.cuda.synchronize()
        for k in OUTS:
            assert torch.equal(s[k].contiguous().view(torch.uint8), eager[k].contiguous().view(torch.uint8)), f"{what}: {k}"
    st = torch.cuda.Stream()
    reset()
    layer_step(mcg, s, T, K, N, stream=st)
    same("another stream")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        layer_step(mcg, s, T, K, N, stream=st)
    for rep in range(3):
        reset()
        g.replay()
        same(f"replay {rep}")
    say(f"  {shape}: same bits on another stream and in three replays")


def test_the_example_learns():
    need_gpu()
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "linear8_layer.py")
    spec = importlib.util.spec_from_file_location("linear8_layer", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses = example.train(T=300, K=512, N=200, steps=12, rate=0.2)
    assert all(b < a for a, b in zip(losses, losses[1:])), losses
