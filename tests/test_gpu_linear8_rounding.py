"""Codes of 8-bit rows at and next to a tie, rows whose squares leave binary32, and the
gradient of rows far from one, against exact values.  Sizes: every form of the row
kernels (rows shorter than a vector, in a wavefront's or a workgroup's registers, and
read twice)."""
import numpy as np
import pytest
import torch

import linear8_ref as ref
from gpu_util import need_gpu
from linear8_ref import DT, U32

pytestmark = pytest.mark.gpu

# rows, columns
FORMS = [(2048, 5), (2048, 8), (300, 300), (300, 700), (300, 1500), (300, 3000), (300, 5000), (40, 8000), (300, 8000),
         (40, 12000), (20, 20000)]


def rows_with_ties(dt, M, N):
    """Rows with the largest values' mantissas in turn (all of them from 1024 rows on for
    f16, 128 for bf16), plus and minus half of it, and values of all sizes below."""
    t = DT[dt]
    bits = 10 if dt == "f16" else 7
    i = torch.arange(M)
    top = (2 ** bits + (i * 37) % 2 ** bits).double() * 2.0 ** (i % 9 - 12).double()
    x = (top[:, None] * torch.from_numpy(np.random.default_rng(N).uniform(-1, 1, (M, N)))).to(t)
    lead = torch.stack([top, top / 2, -top / 2], 1).to(t)
    x[:, :3] = lead
    if N > 8:
        x[:, -3:] = lead
    return x


def exact_quotients(x):
    """127 x / max|x|: a tie is exact in binary64 (127 x and the quotient are), and every
    other quotient of two 16-bit values is at least 2^-20 from one."""
    top = x.double().abs().amax(1, keepdim=True)
    return 127.0 * x.double() / top


@pytest.mark.parametrize("norm", [False, True], ids=["rows", "norm"])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("shape", FORMS, ids=str)
def test_codes_of_16_bit_rows_are_the_nearest(dt, shape, norm):
    mcg = need_gpu()
    M, N = shape
    x = rows_with_ties(dt, M, N)
    X, Q, scale = x.cuda(), torch.empty(M, N, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    if norm:  # without weights and residual the codes do not depend on the norm
        mcg.rmsnorm_quant(dt, M, N, X, N, None, 0, None, 1e-5, None, 0, Q, N, scale)
    else:
        mcg.quantize_rows(dt, M, N, X, N, Q, N, scale)
    want = exact_quotients(x).round()  # ties to even
    bad = Q.cpu().double() != want
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} codes, first at {bad.nonzero()[0].tolist()}"


@pytest.mark.parametrize("shape", FORMS, ids=str)
def test_codes_of_other_rows_are_the_nearest_but_for_roundings(shape):
    mcg = need_gpu()
    M, N = shape
    Q, scale = torch.empty(M, N, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    # binary32: the quotient is rounded to binary32 before it is to an integer
    x = ref.rand(N, M, N, gain=3).float()
    mcg.quantize_rows("f32", M, N, x.cuda(), N, Q, N, scale)
    d = (Q.cpu().double() - exact_quotients(x)).abs().max()
    assert d <= 0.5 + 127 * U32, float(d)
    # a norm of a sum with weights: h and h w (of the value and of the largest) are rounded too
    h, r = ref.rand(N + 1, M, N).to(torch.bfloat16), ref.rand(N + 2, M, N).to(torch.bfloat16)
    w = (1 + 0.2 * ref.rand(N + 3, N)).to(torch.bfloat16)
    mcg.rmsnorm_quant("bf16", M, N, h.cuda(), N, r.cuda(), N, w.cuda(), 1e-5, None, 0, Q, N, scale)
    y = (h.double() + r.double()) * w.double()
    d = (Q.cpu().double() - exact_quotients(y)).abs().max()
    assert d <= 0.5 + 127 * 5 * U32, float(d)


@pytest.mark.parametrize("N", [5, 300, 3000, 12000, 20000])
def test_rows_whose_mean_square_is_below_binary32(N):
    """With eps 0 a row can have a mean square that is no normal binary32 number: it is
    marked like one whose squares overflow.  With an eps it is a row like any other."""
    mcg = need_gpu()
    gains = [1e-42, 1e-36, 1e-25, 1e-21, 1e-18, 1e-3, 1.0]
    M = len(gains) + 1
    x = torch.stack([ref.rand(i, N) for i in range(M)]).float()
    x = x.sign() * x.abs().clamp(0.25, 4.0)
    for i, g in enumerate(gains):
        x[i] = (x[i].double() * g).float()
    x[M - 1] = 0
    Q, scale, rstd = torch.empty(M, N, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    mcg.rmsnorm_quant("f32", M, N, x.cuda(), N, None, 0, None, 0.0, None, 0, Q, N, scale, rstd)
    q, s = Q.cpu(), scale.cpu()
    assert bool(torch.isnan(s[:4]).all()) and not q[:4].any(), s
    assert float(s[M - 1]) == 0 and not q[M - 1].any()
    _, y, rs = ref.rmsnorm(x[4:M - 1], None, None, 0.0)
    top = y.abs().amax(1) / 127
    assert bool(((s[4:M - 1].double() - top).abs() <= 2.0 ** -16 * top).all())
    assert bool(((rstd[4:M - 1].cpu().double() - rs).abs() <= 2.0 ** -17 * rs).all())
    assert bool(((q[4:M - 1].double() - y / top[:, None]).abs() <= 0.5 + 127 * 2 * U32).all())
    mcg.rmsnorm_quant("f32", M, N, x.cuda(), N, None, 0, None, 1e-5, None, 0, Q, N, scale, rstd)
    q, s = Q.cpu(), scale.cpu()
    assert bool(torch.isfinite(s).all()) and bool((q[:M - 1].abs().amax(1) == 127).all())


@pytest.mark.parametrize("x8", [False, True], ids=["x", "x8"])
@pytest.mark.parametrize("N", [5, 300, 700, 1500, 3000, 5000, 8000, 12000, 20000])
def test_gradient_of_rows_far_from_one(N, x8):
    """Rows whose rstd squared is no normal binary32 number (or none at all): the gradient
    is, and is held to the same bound as any row's."""
    mcg = need_gpu()
    gains = [1e-30, 1e-22, 1e-3, 1.0, 1e17, 1e22, 1e30]
    M = len(gains)
    g = torch.tensor(gains, dtype=torch.float64)
    dy = ref.rand(N, M, N).float()
    if x8:
        x, scale = ref.codes(N + 1, M, N), (g * 0.02).float()
        xv = x.double() * scale.double()[:, None]
    else:
        x, scale = (ref.rand(N + 1, M, N) * g[:, None]).float(), None
        xv = x.double()
    rstd = ref.rmsnorm(xv, None, None, 0.0)[2].float()
    dX = torch.empty(M, N, device="cuda")
    mcg.rmsnorm_backward("f32", "i8" if x8 else "f32", M, N, dy.cuda(), N, x.cuda(), N, scale.cuda() if x8 else None, None,
                         rstd.cuda(), None, 0, dX, N, None)
    dx = ref.rmsnorm_backward(dy, xv, None, rstd, None)[0]
    # as in test_rmsnorm_backward of the layer's tests, with binary32 results
    r = rstd.double()[:, None]
    c = r.square() * (dy.double() * xv).abs().mean(1, keepdim=True)
    tol = (64 + N // 1024) * U32 * r * (dy.double().abs() + c * xv.abs()) + U32 * dx.abs() + ref.SUB["f32"]
    d = (dX.cpu().double() - dx).abs()
    ok = d <= tol
    assert bool(ok.all()), [(gains[i], float((d[i] / tol[i]).nan_to_num(1e30).max())) for i in range(M) if not bool(ok[i].all())]
