"""Plain binary64 forms of the 8-bit linear layer's operators, for its tests."""
import numpy as np
import torch

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
# a rounding to the type is off by at most half a step: U relative to the value,
# and half the spacing near zero (SUB)
U = {k: torch.finfo(t).eps / 2 for k, t in DT.items()}
SUB = {k: float(torch.finfo(t).smallest_normal) * torch.finfo(t).eps / 2 for k, t in DT.items()}
U32 = 2.0 ** -24


def rmsnorm(x, r, w, eps):
    """h, y, rstd in binary64."""
    h = x.double() if r is None else x.double() + r.double()
    rstd = (h.square().mean(1) + eps).rsqrt()
    y = h * rstd[:, None]
    return h, (y if w is None else y * w.double()), rstd


def rmsnorm_backward(dy, x, w, rstd, dr):
    """dx, dw in binary64 with rstd as given."""
    dy, x, rstd = dy.double(), x.double(), rstd.double()[:, None]
    g = dy if w is None else dy * w.double()
    dx = rstd * (g - x * rstd.square() * (g * x).mean(1, keepdim=True))
    if dr is not None:
        dx = dx + dr.double()
    return dx, (dy * x * rstd).sum(0)


def i8_scaled(a, sa, b, sb, bias):
    """b as K x N; the integer products are exact in binary64."""
    d = (a.double() @ b.double()) * sa.double()[:, None] * sb.double()
    return d if bias is None else d + bias.double()


def grad_i8(a, q, s, c, beta):
    """D and the sum of the products' magnitudes; a as M x K."""
    v = q.double() * s.double()[:, None]
    d = a.double() @ v
    mag = a.double().abs() @ v.abs()
    return (d if c is None else d + beta * c.double()), mag


def strided(rows, cols, pad, dtype, device="cpu", offset=0):
    """A rows x cols view whose rows lie cols + pad elements apart and start
    `offset` elements into the buffer, with NaN patterns around it."""
    n = rows * (cols + pad) + offset + 8
    if dtype == torch.int8:
        buf = torch.full((n,), -77, dtype=dtype, device=device)
    else:
        buf = torch.full((n,), float("nan"), dtype=dtype, device=device)
    return buf[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]


def around(view, rows, cols):
    """What lies between the rows of a strided() view, as bytes."""
    return view.as_strided((rows, view.stride(0)), view.stride())[:, cols:].contiguous().view(torch.uint8)


def fill(view, values):
    view.copy_(values.to(view.dtype))
    return view


def rand(seed, *shape, gain=1.0):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape)) * gain


def codes(seed, *shape):
    return torch.from_numpy(np.random.default_rng(seed).integers(-127, 128, shape).astype(np.int8))
