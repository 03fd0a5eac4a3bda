"""The plain forms that the 8-bit linear layer is tested against: their gradients
against central differences, and the checks against planted mistakes."""
import torch

import linear8_ref as ref


def test_norm_gradient_against_differences():
    M, N, eps = 3, 11, 1e-5
    x, w, dy = ref.rand(1, M, N), 1 + 0.3 * ref.rand(2, N), ref.rand(3, M, N)
    dr = ref.rand(4, M, N)

    def loss(x, w):
        h, y, _ = ref.rmsnorm(x, None, w, eps)
        return (y * dy).sum() + (h * dr).sum()
    rstd = ref.rmsnorm(x, None, w, eps)[2]
    dx, dw = ref.rmsnorm_backward(dy, x, w, rstd, dr)
    e = 1e-5
    for i in range(M):
        for j in range(N):
            d = torch.zeros_like(x)
            d[i, j] = e
            # central differences: truncation e^2 times a third derivative of order 1, and 1e-16 / e of rounding
            assert abs((loss(x + d, w) - loss(x - d, w)) / (2 * e) - dx[i, j]) < 1e-8
    for j in range(N):
        d = torch.zeros_like(w)
        d[j] = e
        assert abs((loss(x, w + d) - loss(x, w - d)) / (2 * e) - dw[j]) < 1e-8


def test_linear_gradients_against_differences():
    # y = x . W^T with x and W in 8 bits: the gradients that gemm_grad_i8 forms
    T, K, N = 5, 7, 6
    qx, sx, qw, sw = ref.codes(1, T, K), ref.rand(2, T).abs(), ref.codes(3, N, K), ref.rand(4, N).abs()
    x, w, dy = qx.double() * sx[:, None], qw.double() * sw[:, None], ref.rand(5, T, N)
    dw, _ = ref.grad_i8(dy.T, qx, sx, None, 0)
    dx, _ = ref.grad_i8(dy, qw, sw, None, 0)
    loss = lambda x, w: ((x @ w.T) * dy).sum()
    e = 1e-3  # the loss is linear in each argument: only rounding is left, 1e-16 * |loss| / e
    tol = 1e-15 * float((x.abs() @ w.abs().T * dy.abs()).sum()) / e
    for i in range(N):
        for j in range(K):
            d = torch.zeros_like(w)
            d[i, j] = e
            assert abs((loss(x, w + d) - loss(x, w - d)) / (2 * e) - dw[i, j]) < tol
    for i in range(T):
        for j in range(K):
            d = torch.zeros_like(x)
            d[i, j] = e
            assert abs((loss(x + d, w) - loss(x - d, w)) / (2 * e) - dx[i, j]) < tol


def test_a_norm_without_its_mean_term_is_told_apart():
    x, dy = ref.rand(1, 4, 64), ref.rand(2, 4, 64)
    rstd = ref.rmsnorm(x, None, None, 1e-5)[2]
    dx, _ = ref.rmsnorm_backward(dy, x, None, rstd, None)
    wrong = rstd[:, None] * dy
    assert float((dx - wrong).abs().max()) > 100 * ref.U["bf16"]


def test_strided_views_hold_their_surroundings():
    v = ref.strided(3, 5, 2, torch.float32, offset=1)
    ref.fill(v, torch.ones(3, 5))
    assert v.stride() == (7, 1) and bool(torch.isnan(v.as_strided((3, 7), (7, 1))[:, 5:]).all())
    assert ref.around(v, 3, 5).numel() == 3 * 2 * 4
