"""Products of the 8-bit linear layer that run each form of its kernels, with what their
plans say of them (include/mcg.h, mcg_i8_scaled_path).  tests/test_linear8_plans.py holds
the plans to this table on the host, tests/test_gpu_linear8_forms.py runs them."""
import torch

import linear8_ref as ref
from linear8_ref import DT, SUB, U, U32

GENERAL, FAST, STREAM, MID, HALF = 0, 1, 4, 6, 7
MIB = 1 << 20


def up(x, y):
    return -(-x // y) * y


# layoutB, M, N, K, operands with 16-byte rows, workspace, kernel, panels, stream-K tiles, K ranges
SCALED = [
    # stream-K with 128 x 128 tiles: nothing but pieces, and pieces after whole rounds
    ("k_contig", 93, 1216, 8128, True, 64 * MIB, MID, 0, 10, 1),
    ("mn_contig", 93, 1216, 8128, True, 64 * MIB, MID, 0, 10, 1),
    ("k_contig", 376, 251, 4000, True, 64 * MIB, MID, 0, 6, 1),
    ("mn_contig", 991, 109, 3984, True, 64 * MIB, MID, 0, 8, 1),
    ("k_contig", 2997, 1310, 3520, True, 64 * MIB, MID, 0, 8, 1),
    ("mn_contig", 2772, 1454, 3504, True, 64 * MIB, MID, 0, 8, 1),
    # with 256 x 256 tiles
    ("k_contig", 7199, 2207, 2496, True, 64 * MIB, FAST, 0, 5, 1),
    ("mn_contig", 2273, 7203, 2448, True, 64 * MIB, FAST, 0, 5, 1),
    # on copies of operands without 16-byte rows
    ("k_contig", 884, 860, 6496, False, 64 * MIB, MID, 1, 49, 1),
    ("mn_contig", 1002, 743, 6608, False, 64 * MIB, MID, 1, 48, 1),
    ("k_contig", 7293, 2267, 2448, False, 64 * MIB, FAST, 1, 5, 1),
    ("mn_contig", 7290, 2232, 2512, False, 64 * MIB, FAST, 1, 5, 1),
    # panels cut along N, the last one narrower
    ("k_contig", 816, 883, 3456, False, 5031936, HALF, 2, 0, 1),
    ("mn_contig", 376, 1456, 3088, False, 4125568, HALF, 2, 0, 1),
    ("k_contig", 2825, 1445, 4144, False, 15685040, MID, 2, 0, 1),
    ("mn_contig", 3331, 1155, 4384, False, 18811744, MID, 2, 0, 1),
    ("k_contig", 5403, 1471, 6176, False, 39297888, MID, 2, 2, 1),
    ("mn_contig", 5407, 1509, 6832, False, 43499344, MID, 2, 2, 1),
    # the streaming kernel with blocks of 128 columns of K-contiguous weights, K whole and cut
    ("k_contig", 24, 16500, 512, True, 0, STREAM, 0, 0, 1),
    ("k_contig", 1, 16421, 4096, True, 0, STREAM, 0, 0, 1),
    ("k_contig", 7, 16421, 4096, True, 64 * MIB, STREAM, 0, 0, 3),
]


def scaled_lds(layout, M, N, K, aligned):
    """Leading dimensions of A and B."""
    cols = K if layout == "k_contig" else N
    return (up(K, 16), up(cols, 16)) if aligned else (K + 5, cols + 7)


# D's type (A f16 and bf16 plan alike), layoutA, M, N, K, A with 16-byte rows, workspace, kernel, panels, stream-K tiles
GRAD = [
    ("f32", "k_contig", 256, 251, 640, True, 0, GENERAL, 0, 0),
    ("f32", "mn_contig", 131, 300, 515, False, 0, GENERAL, 0, 0),
    ("16", "k_contig", 416, 277, 1448, True, 806912, HALF, 2, 0),
    ("16", "mn_contig", 436, 274, 1672, True, 921600, HALF, 2, 0),
    ("16", "mn_contig", 357, 1324, 1696, False, 3046160, HALF, 2, 0),
    ("16", "k_contig", 4695, 814, 1280, True, 1376256, MID, 2, 0),
    ("f32", "k_contig", 893, 642, 280, True, 64 * MIB, HALF, 1, 0),
    ("f32", "mn_contig", 1549, 386, 272, False, 64 * MIB, HALF, 1, 0),
    ("f32", "k_contig", 4721, 787, 776, True, 1654784, MID, 2, 0),
    ("f32", "mn_contig", 2349, 1965, 792, False, 4647744, MID, 2, 0),
    ("f32", "mn_contig", 4221, 4882, 328, False, 3579168, FAST, 2, 0),
    ("f32", "k_contig", 3308, 3801, 64, True, 64 * MIB, FAST, 1, 0),
    ("16", "k_contig", 3394, 3890, 72, True, 64 * MIB, FAST, 1, 0),
    ("16", "mn_contig", 1893, 4744, 136, False, 64 * MIB, FAST, 1, 0),
    ("16", "k_contig", 2481, 127, 2872, True, 64 * MIB, MID, 1, 20),
    ("16", "mn_contig", 877, 424, 3176, False, 64 * MIB, MID, 1, 28),
    ("16", "k_contig", 3531, 4770, 1480, True, 64 * MIB, FAST, 1, 10),
    ("f32", "k_contig", 3658, 1100, 1744, True, 64 * MIB, MID, 1, 5),
    ("f32", "mn_contig", 2763, 1428, 1744, False, 64 * MIB, MID, 1, 8),
    ("f32", "mn_contig", 4711, 3468, 1496, True, 64 * MIB, FAST, 1, 10),
]


def grad_lda(layout, M, K, aligned):
    cols = K if layout == "k_contig" else M
    return up(cols, 8) if aligned else cols + 3


def few_nonzeros(seed, M, K, n, dt):
    """An M x K matrix with n nonzeros in every row, of one magnitude's order."""
    g = torch.Generator().manual_seed(seed)
    a = torch.zeros(M, K, dtype=DT[dt])
    k = torch.stack([torch.randperm(K, generator=g)[:n] for _ in range(M)]) if M <= 64 else torch.randint(0, K, (M, n), generator=g)
    v = (0.5 + torch.rand(M, n, generator=g)) * (torch.randint(0, 2, (M, n), generator=g) * 2 - 1)
    return a.scatter_(1, k, v.to(DT[dt]))


def sparse_grad_tol(dt, a, d, mag, n):
    """For a binary32 result and n nonzeros a row: s q is formed with one binary32 rounding
    and taken as two values of A's type, which leaves U^2 of it (and half the spacing near
    zero); 2 n products are added on the matrix cores (4 u per addition, as in the layer's
    other bounds; adding zeros is exact), and the two sums to one result."""
    return (U[dt] ** 2 + (1 + 4 * (2 * n + 2)) * U32) * mag + SUB[dt] * a.double().abs().sum(1, keepdim=True) + 2 * U32 * d.abs()


def split_values(q, s, dt):
    """The two values of A's type that stand for s q (binary32), as the kernels form them."""
    v = q.float() * s[:, None]
    hi = v.to(DT[dt])
    return hi.double(), (v - hi.float()).to(DT[dt]).double()


def grad_inputs(seed, K, N):
    return ref.codes(seed, K, N), ref.rand(seed + 1, K).abs().float() * 0.02 + 1e-3
