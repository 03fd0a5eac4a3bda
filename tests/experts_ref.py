"""Plain binary64 forms of the products by group and of block-scaled 8-bit floats, for
their tests, and the bounds that the kernels' roundings allow."""
import numpy as np
import torch

from linear8_ref import DT, SUB, U, U32, rand, strided  # noqa: F401

F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
BLOCK = 128
KINDS = {"1x128": (1, 128), "128x1": (128, 1), "128x128": (128, 128)}


def cdiv(a, b):
    return -(-a // b)


def per_element(s, m, n, bm, bn):
    """Each block's value at every element."""
    return s.repeat_interleave(bm, -2)[..., :m, :].repeat_interleave(bn, -1)[..., :n]


def block_max(x, bm, bn):
    m, n = x.shape
    out = torch.empty(cdiv(m, bm), cdiv(n, bn), dtype=x.dtype)
    for i in range(out.shape[0]):
        for j in range(out.shape[1]):
            out[i, j] = x[i * bm:(i + 1) * bm, j * bn:(j + 1) * bn].abs().max()
    return out


def to_f8(y, to):
    """The nearest 8-bit floats of binary32 values within the format's range, ties to even."""
    return y.to(F8[to]).view(torch.uint8)


def quantize(x, to, bm, bn):
    """Codes (uint8) and binary32 scales of finite x: L x and its quotient are rounded to
    binary32 (taken in binary64 here, where neither overflows; the quotient of two
    binary32 values rounded twice is that rounded once, since binary64 has more than
    twice its bits)."""
    x = x.float()
    top = block_max(x, bm, bn)
    lx = (x.double() * LARGEST[to])
    huge = per_element((top >= 2.0 ** 64).double() * 2.0 ** -64 + (top < 2.0 ** 64).double(), *x.shape, bm, bn)
    tiny = per_element((top < 2.0 ** -64).double() * 2.0 ** 64 + (top >= 2.0 ** -64).double(), *x.shape, bm, bn)
    lx = (lx * huge * tiny).float().double()
    t = per_element(top, *x.shape, bm, bn).double() * huge * tiny
    y = torch.where(t > 0, lx / t, torch.zeros_like(lx)).float()
    return to_f8(y, to), (top.double() / LARGEST[to]).float()


def values(codes, to, scale, bm, bn):
    """In binary64."""
    q = codes.view(F8[to]).double()
    return q * per_element(scale.double(), *codes.shape[-2:], bm, bn)


def random_codes(seed, m, n, to, bm, bn, gain=1.0):
    """Codes and scales of normal rows whose magnitudes differ from block to block."""
    x = rand(seed, m, n, gain=gain)
    s = torch.exp(0.7 * rand(seed + 1, cdiv(m, bm), cdiv(n, bn)))
    return quantize((x * per_element(s, m, n, bm, bn)).float(), to, bm, bn)


def offsets_of(sizes, first=0):
    return torch.tensor([first + sum(sizes[:i]) for i in range(len(sizes) + 1)], dtype=torch.int32)


def grouped(a, b, offsets):
    """D and the sum of the products' magnitudes, by rows; b: G matrices K x N.  NaN in the
    rows of no group."""
    a, b = a.double(), b.double()
    d = torch.full((a.shape[0], b.shape[2]), float("nan"), dtype=torch.float64)
    mag = d.clone()
    for g, (r0, r1) in enumerate(zip(offsets.tolist(), offsets.tolist()[1:])):
        d[r0:r1] = a[r0:r1] @ b[g]
        mag[r0:r1] = a[r0:r1].abs() @ b[g].abs()
    return d, mag


def grouped_grad(a, b, offsets, c, beta):
    a, b = a.double(), b.double()
    G = len(offsets) - 1
    d = torch.zeros(G, a.shape[1], b.shape[1], dtype=torch.float64)
    mag = d.clone()
    for g, (r0, r1) in enumerate(zip(offsets.tolist(), offsets.tolist()[1:])):
        d[g] = a[r0:r1].T @ b[r0:r1]
        mag[g] = a[r0:r1].abs().T @ b[r0:r1].abs()
    return (d if c is None else d + beta * c.double()), mag


def tol_16(d, mag, K, dtD):
    """The dense products' bound, 4 u (K + 2) sum|ab|, and the rounding to D's type (of a
    value that may be off by that bound already), C's product and sum among it."""
    acc = 4 * U32 * (K + 2) * mag
    return acc + (U[dtD] + 2 * U32) * (d.abs() + acc) + SUB[dtD]


def tol_f8(d, mag, K, dtD):
    """Within a block the dense products' bound over 128 values, or 2^-10 of the sum of the
    magnitudes more on the 8-bit instructions (bf16 D); then the product of the scales,
    its product with the sum and the sum over the blocks, a rounding each."""
    acc = ((4 * 130 + cdiv(K, BLOCK) + 3) * U32 + (2.0 ** -10 if dtD == "bf16" else 0.0)) * mag
    return acc + (U[dtD] + 2 * U32) * (d.abs() + acc) + SUB[dtD]
