"""GPU parity of the products by group and of block-scaled 8-bit floats with their
plain binary64 forms: every type, layout, kernel, odd and strided operands, empty and
uneven groups, rows of no group, values that are no numbers, streams and graphs.
Tolerances count roundings (experts_ref)."""
import numpy as np
import pytest
import torch

import experts_cases as cases
import experts_ref as ref
from experts_ref import BLOCK, DT, F8, KINDS, cdiv
from gpu_util import need_gpu, say

pytestmark = pytest.mark.gpu
GUARD8 = 0x5A  # what lies around 8-bit rows


def buf(rows, cols, dtype, pad=0, offset=0):
    """A rows x cols view in a buffer with guards around and between the rows."""
    n = rows * (cols + pad) + offset + 16
    fill = GUARD8 if dtype == torch.uint8 else float("nan")
    b = torch.full((n,), fill, dtype=dtype, device="cuda")
    return b[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]


def put(t, pad=0, offset=0):
    v = buf(t.shape[0], t.shape[1], t.dtype, pad, offset)
    v.copy_(t)
    return v


def put3(t, pad=0, gap=0, offset=0):
    """G matrices of one buffer, each `gap` elements behind the one before."""
    G, r, c = t.shape
    stride = r * (c + pad) + gap
    fill = GUARD8 if t.dtype == torch.uint8 else float("nan")
    b = torch.full((offset + G * stride + 16,), fill, dtype=t.dtype, device="cuda")
    v = b.as_strided((G, r, c), (stride, c + pad, 1), offset)
    v.copy_(t)
    return v


def ld(t):
    return 0 if t is None else t.stride(-2)


def guards_hold(*views):
    """Nothing was written outside the views."""
    torch.cuda.synchronize()
    for v in views:
        if v is None:
            continue
        base = v._base if v._base is not None else v
        flat = base.as_strided((base.untyped_storage().nbytes() // base.element_size(),), (1,), 0)
        mine = torch.zeros_like(flat, dtype=torch.bool)
        mine.as_strided(v.shape, v.stride(), v.storage_offset()).fill_(True)
        rest = flat[~mine]
        assert bool((rest == GUARD8).all() if v.dtype == torch.uint8 else torch.isnan(rest).all()), "wrote outside its rows"


def within(got, exact, tol, what):
    d = (got.double().cpu() - exact).abs()
    bad = ~(d <= tol)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {float((d / tol).nan_to_num(1e30).max())} of the tolerance"


# ------------------------------------------------------------------ blocks
BLOCK_SHAPES = [(1, 1), (3, 7), (2, 8), (1, 129), (17, 128), (130, 127), (128, 128), (129, 257), (300, 1000), (5, 4096), (257, 2047)]


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("to", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_blocks(dt, to, kind):
    """Codes, scales and values bit for bit."""
    mcg = need_gpu()
    bm, bn = KINDS[kind]
    for M, N in BLOCK_SHAPES:
        for pad, off in ((0, 0), (3, 1)):
            x = (ref.rand(M * 31 + N, M, N) * torch.exp(ref.rand(N, N))).to(DT[dt])
            q, scale = ref.quantize(x, to, bm, bn)
            X, Q = put(x, pad, off), buf(M, N, torch.uint8, pad, off)
            S = buf(cdiv(M, bm), cdiv(N, bn), torch.float32, pad)
            mcg.quantize_blocks(dt, to, bm, bn, M, N, X, ld(X), Q, ld(Q), S, ld(S))
            guards_hold(Q, S)
            assert torch.equal(S.cpu(), scale), f"scales {M} x {N}"
            assert torch.equal(Q.cpu(), q), f"codes {M} x {N}: {int((Q.cpu() != q).sum())} differ"
            for dtD in ("bf16", "f16", "f32"):
                D = buf(M, N, DT[dtD], pad, off)
                mcg.dequantize_blocks(to, dtD, bm, bn, M, N, Q, ld(Q), S, ld(S), D, ld(D))
                guards_hold(D)
                v = (q.view(F8[to]).float() * ref.per_element(scale, M, N, bm, bn)).to(DT[dtD])
                assert torch.equal(D.cpu(), v), f"values {M} x {N} {dtD}"


@pytest.mark.parametrize("dt,to", [("bf16", "e4m3"), ("f16", "e5m2"), ("f32", "e4m3")])
def test_blocks_of_many_rows(dt, to):
    """1 x 128 blocks with more rows in a thread (over 1024 workgroups of 64 rows x 128 columns)."""
    mcg = need_gpu()
    M, N = 7003, 1187
    x = (ref.rand(5, M, N) * torch.exp(ref.rand(6, N))).to(DT[dt])
    x[M - 1, N - 1], x[70, 130] = float("inf"), float("nan")
    X, Q, S = put(x, 5, 1), buf(M, N, torch.uint8, 5, 1), buf(M, cdiv(N, BLOCK), torch.float32, 1)
    mcg.quantize_blocks(dt, to, 1, BLOCK, M, N, X, ld(X), Q, ld(Q), S, ld(S))
    guards_hold(Q, S)
    for r, c in ((M - 1, 9), (70, 1)):  # no numbers: scale NaN, codes 0
        assert bool(torch.isnan(S[r, c])) and not bool(Q[r, BLOCK * c:BLOCK * (c + 1)].any())
        x[r, BLOCK * c:BLOCK * (c + 1)] = 0
        S[r, c] = 0
    q, scale = ref.quantize(x, to, 1, BLOCK)
    assert torch.equal(S.cpu(), scale) and torch.equal(Q.cpu(), q)


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("to", ["e4m3", "e5m2"])
def test_blocks_of_nothing_and_of_no_number(to, kind):
    mcg = need_gpu()
    bm, bn = KINDS[kind]
    M, N = 9 * bm, 3 * bn if bn > 1 else 20
    x = ref.rand(1, M, N).float()
    rows = [x[i * bm:(i + 1) * bm] for i in range(9)]
    rows[0].zero_()
    rows[1].fill_(-0.0)
    rows[2][0, 0] = float("nan")
    rows[3][-1, -1] = float("inf")
    rows[4][0, 1] = float("-inf")
    rows[5].mul_(1e-42)   # subnormal values
    rows[6].mul_(1e-30)
    rows[7].mul_(3e37)    # L x leaves binary32
    X, Q, S = put(x), buf(M, N, torch.uint8), buf(cdiv(M, bm), cdiv(N, bn), torch.float32)
    mcg.quantize_blocks("f32", to, bm, bn, M, N, X, ld(X), Q, ld(Q), S, ld(S))
    torch.cuda.synchronize()
    top = ref.block_max(torch.where(torch.isfinite(x), x, torch.full_like(x, float("inf"))), bm, bn)
    bad = ~torch.isfinite(top)
    assert int(bad.sum()) == 3
    q, scale = ref.quantize(torch.where(ref.per_element(bad, M, N, bm, bn), torch.zeros_like(x), x), to, bm, bn)
    assert bool(torch.isnan(S.cpu())[bad].all()) and torch.equal(S.cpu()[~bad], scale[~bad])
    assert torch.equal(Q.cpu() & 0x7F, q & 0x7F)
    D = buf(M, N, torch.float32)
    mcg.dequantize_blocks(to, "f32", bm, bn, M, N, Q, ld(Q), S, ld(S), D, ld(D))
    assert torch.equal(torch.isnan(D.cpu()), ref.per_element(bad, M, N, bm, bn))


def test_every_code_is_read_as_its_value():
    mcg = need_gpu()
    q = torch.arange(256, dtype=torch.uint8)[None]
    for to in F8:
        D, s = buf(1, 256, torch.float32), torch.tensor([[1.0, 0.5]], device="cuda")
        mcg.dequantize_blocks(to, "f32", 1, 128, 1, 256, q.cuda(), 256, s, 2, D, 256)
        v = q.view(F8[to]).float() * torch.tensor([1.0] * 128 + [0.5] * 128)
        assert torch.equal(torch.nan_to_num(D.cpu(), nan=777.0), torch.nan_to_num(v, nan=777.0))


# ----------------------------------------------------------------- grouped
SIZES = {"one": [37], "even": [16, 16, 16, 16], "uneven": [1, 0, 130, 7, 0, 0, 64, 300], "empty": [0, 0, 0],
         "single": [1] * 70, "many": [(i * 7) % 5 for i in range(150)], "last": [0] * 5 + [200], "large": [257, 600, 3, 1030]}
PADS = [(0, 0), (5, 1), (8, 0)]  # elements between rows, and before the first


def run_grouped(mcg, dt, lb, a, b, off, dtD, pad=0, first=0, gap=0, stream=None):
    """Returns D (with NaN wherever nothing was written)."""
    M, K = a.shape
    G, _, N = b.shape
    A = put(a.to(DT[dt]), pad, first)
    B = put3((b if lb == "mn_contig" else b.transpose(1, 2).contiguous()).to(DT[dt]), pad, gap, first)
    D = buf(M, N, DT[dtD], pad, first)
    mcg.gemm_grouped(dt, lb, G, M, N, K, off.cuda(), A, ld(A), B, ld(B), B.stride(0), D, ld(D), dtD, stream)
    guards_hold(D)
    return D


def check_grouped(mcg, dt, lb, dtD, sizes, N, K, pad, first, lead=0, tail=0, gap=0):
    M = lead + sum(sizes) + tail
    a = ref.rand(M * 7 + K, M, K).to(DT[dt])
    a[:lead] = float("nan")
    a[M - tail:] = float("nan")
    b = (ref.rand(N + 1, len(sizes), K, N) / max(K, 1) ** 0.5).to(DT[dt])
    off = ref.offsets_of(sizes, lead)
    D = run_grouped(mcg, dt, lb, a, b, off, dtD, pad, first, gap).cpu()
    d, mag = ref.grouped(a, b.double(), off)
    inside = slice(lead, M - tail)
    assert bool(torch.isnan(D[:lead]).all()) and bool(torch.isnan(D[M - tail:]).all()), "wrote rows of no group"
    within(D[inside], d[inside], ref.tol_16(d[inside], mag[inside], K, dtD), f"{dt} {lb} {dtD} {sizes} {N} x {K} pad {pad}")


@pytest.mark.parametrize("sizes", list(SIZES))
@pytest.mark.parametrize("lb", ["k_contig", "mn_contig"])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_gemm_grouped(dt, lb, sizes):
    mcg = need_gpu()
    for (N, K), (pad, first) in zip([(64, 64), (128, 200), (200, 72), (129, 130), (8, 512), (300, 1000), (5, 3), (40, 1)],
                                    PADS * 3):
        for dtD in (dt, "f32"):
            check_grouped(mcg, dt, lb, dtD, SIZES[sizes], N, K, pad, first, lead=2 * (pad > 0), tail=3, gap=pad)


@pytest.mark.parametrize("lb", ["k_contig", "mn_contig"])
@pytest.mark.parametrize("shape", [([900, 0, 1100, 250], 512, 512), ([300, 200, 290, 310, 100], 768, 640),
                                   ([70, 50, 64, 128, 90, 1], 384, 1024), ([10, 3, 20, 0, 17, 33], 1024, 768),
                                   ([1, 1, 2, 1], 2048, 2048), ([129] * 40, 256, 256)], ids=str)
def test_gemm_grouped_of_larger_sizes(lb, shape):
    """Aligned operands of the sizes that the faster kernels take."""
    mcg = need_gpu()
    sizes, N, K = shape
    for dt, dtD in (("bf16", "bf16"), ("f16", "f32")):
        check_grouped(mcg, dt, lb, dtD, sizes, N, K, 0, 0, lead=5, tail=70)
        check_grouped(mcg, dt, lb, dtD, sizes, N + 24, K + 40, 8, 0, tail=1, gap=16)


def test_gemm_grouped_with_shared_weights_and_no_k():
    mcg = need_gpu()
    a, b = ref.rand(1, 50, 64).bfloat16(), ref.rand(2, 1, 64, 48).bfloat16()
    off = ref.offsets_of([20, 0, 30])
    A, B, D = put(a), put(b[0]), buf(50, 48, torch.float32)
    mcg.gemm_grouped("bf16", "mn_contig", 3, 50, 48, 64, off.cuda(), A, 64, B, 48, 0, D, 48, "f32")
    d, mag = ref.grouped(a, b.double().expand(3, -1, -1), off)
    within(D, d, ref.tol_16(d, mag, 64, "f32"), "shared weights")
    D = buf(50, 48, torch.bfloat16)
    off = ref.offsets_of([20, 0, 10], first=4)
    mcg.gemm_grouped("bf16", "k_contig", 3, 50, 48, 0, off.cuda(), None, 1, None, 1, 0, D, 48, "bf16")
    torch.cuda.synchronize()
    assert not bool(D[4:34].any()) and bool(torch.isnan(D[:4]).all()) and bool(torch.isnan(D[34:]).all())


def test_gemm_grouped_keeps_values_that_are_no_numbers_in_their_rows():
    mcg = need_gpu()
    for N, K, sizes in ((256, 256, [100, 300, 60]), (64, 72, [3, 0, 40]), (130, 66, [20, 50]), (512, 256, [2, 1, 3])):
        M = sum(sizes)
        a, b = ref.rand(1, M, K).bfloat16(), ref.rand(2, len(sizes), N, K).bfloat16()
        off = ref.offsets_of(sizes)
        a[1, 3], a[M - 1, K - 1] = float("nan"), float("inf")
        b[-1, 2, 5] = float("nan")  # one weight of the last group
        D = run_grouped(mcg, "bf16", "k_contig", a, b.transpose(1, 2), off, "bf16").cpu()
        bad = torch.zeros(M, N, dtype=torch.bool)
        bad[1], bad[M - 1] = True, True
        bad[off[-2]:, 2] = True
        assert torch.equal(~torch.isfinite(D), bad), (N, K, sizes)


# ------------------------------------------------------------ grouped_grad
def check_grad(mcg, dt, dtD, sizes, M, N, pad, first, beta, lead=0, tail=0, alias=False):
    K, G = lead + sum(sizes) + tail, len(sizes)
    a, b = ref.rand(M + 1, K, M).to(DT[dt]), ref.rand(N + 2, K, N).to(DT[dt])
    for t in (a, b):
        t[:lead] = float("nan")
        t[K - tail:] = float("nan")
    c = ref.rand(5, G, M, N).to(DT[dtD]) if beta else None
    off = ref.offsets_of(sizes, lead)
    A, B = put(a, pad, first), put(b, pad, first)
    D = put3(c if alias else torch.full((G, M, N), float("nan"), dtype=DT[dtD]), pad, pad, first)
    C = None if c is None else D if alias else put3(c, pad, pad, first)
    mcg.gemm_grouped_grad(dt, G, M, N, K, off.cuda(), A, ld(A), B, ld(B), C, D, ld(D), D.stride(0), dtD, beta)
    guards_hold(D)
    d, mag = ref.grouped_grad(a, b, off, c, beta)
    longest = max(sizes, default=0)
    mag = mag if c is None else mag + c.double().abs() * abs(beta)
    within(D, d, ref.tol_16(d, mag, longest, dtD), f"{dt} {dtD} {sizes} {M} x {N} pad {pad} beta {beta}")


@pytest.mark.parametrize("sizes", list(SIZES))
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_gemm_grouped_grad(dt, sizes):
    mcg = need_gpu()
    few = SIZES[sizes] if sizes not in ("single", "many") else SIZES[sizes][:30]
    for (M, N), (pad, first) in zip([(64, 64), (128, 200), (200, 72), (129, 130), (8, 256), (5, 40), (3, 2)], PADS * 3):
        for dtD, beta, alias in ((dt, 0.0, False), ("f32", 0.0, False), ("f32", 1.0, True), (dt, -0.5, False)):
            check_grad(mcg, dt, dtD, few, M, N, pad, first, beta, lead=pad, tail=3, alias=alias)


@pytest.mark.parametrize("shape", [([900, 0, 1100, 250], 512, 512), ([300, 1, 290, 64, 100], 768, 640), ([2000], 1024, 256),
                                   ([0, 0, 7], 256, 264)], ids=str)
def test_gemm_grouped_grad_of_larger_sizes(shape):
    mcg = need_gpu()
    sizes, M, N = shape
    for dt, dtD, beta in (("bf16", "bf16", 0.0), ("f16", "f32", 1.0)):
        check_grad(mcg, dt, dtD, sizes, M, N, 0, 0, beta, tail=40)
        check_grad(mcg, dt, dtD, sizes, M + 24, N + 8, 8, 0, beta, lead=3)


def test_gemm_grouped_grad_without_rows():
    mcg = need_gpu()
    c = ref.rand(1, 2, 40, 48).float()
    for beta in (0.0, 2.0):
        D = put3(torch.full((2, 40, 48), float("nan")))
        C = put3(c)
        mcg.gemm_grouped_grad("bf16", 2, 40, 48, 0, None, None, 40, None, 48, C if beta else None, D, 48, D.stride(0), "f32", beta)
        torch.cuda.synchronize()
        assert torch.equal(D.cpu(), beta * c)


# --------------------------------------------------------------- f8 blocks
def f8_operand(seed, layout, mn, K, to, bmn, gain=1.0):
    """Codes and scales as they are stored, and the binary64 values mn x K."""
    if layout == "k_contig":
        q, s = ref.random_codes(seed, mn, K, to, bmn, BLOCK, gain)
        return q, s, ref.values(q, to, s, bmn, BLOCK)
    q, s = ref.random_codes(seed, K, mn, to, BLOCK, bmn, gain)
    return q, s, ref.values(q, to, s, BLOCK, bmn).T


def check_f8(mcg, to, la, lb, bb, M, N, K, dtD, pad=0, first=0, beta=0.0, alias=False):
    qa, sa, a = f8_operand(M + 11, la, M, K, to, 1)
    qb, sb, b = f8_operand(N + 13, lb, N, K, "e4m3", bb, max(K, 1) ** -0.5)
    A, B, SA, SB = put(qa, pad, first), put(qb, pad, first), put(sa, pad), put(sb, pad, first)
    c = ref.rand(3, M, N).to(DT[dtD]) if beta else None
    D = put(c, pad, first) if alias else buf(M, N, DT[dtD], pad, first)
    C = None if c is None else D if alias else put(c, pad, first)
    mcg.gemm_f8_blocks(to, "e4m3", la, lb, bb, M, N, K, A, ld(A), SA, ld(SA), B, ld(B), SB, ld(SB), C, D, ld(D), dtD, beta)
    guards_hold(D)
    d, mag = a @ b.T, a.abs() @ b.abs().T
    if c is not None:
        d, mag = d + beta * c.double(), mag + abs(beta) * c.double().abs()
    within(D, d, ref.tol_f8(d, mag, K, dtD), f"{to} {la} {lb} {bb} {M} x {N} x {K} {dtD} pad {pad} beta {beta}")


LAYOUTS = ["k_contig", "mn_contig"]


@pytest.mark.parametrize("bb", [1, 128])
@pytest.mark.parametrize("lb", LAYOUTS)
@pytest.mark.parametrize("la", LAYOUTS)
def test_gemm_f8_blocks(la, lb, bb):
    mcg = need_gpu()
    shapes = [(1, 1, 1), (1, 128, 128), (5, 130, 129), (33, 64, 640), (64, 200, 16), (100, 257, 300), (129, 128, 1000), (7, 300, 128)]
    for i, (M, N, K) in enumerate(shapes):
        pad, first = PADS[i % 3] if i % 3 != 2 else (16, 0)
        to = "e5m2" if i % 2 else "e4m3"
        for dtD in ("bf16", "f16", "f32"):
            check_f8(mcg, to, la, lb, bb, M, N, K, dtD, pad, first)
        check_f8(mcg, to, la, lb, bb, M, N, K, "f32", pad, first, beta=1.0, alias=True)


@pytest.mark.parametrize("shape", [(1, 512, 1024), (17, 400, 2048), (64, 384, 512), (300, 272, 784), (256, 512, 384), (700, 1040, 1152),
                                   (1024, 768, 256)], ids=str)
@pytest.mark.parametrize("kind", ["out", "dx", "dw", "rows", "mixed"])
def test_gemm_f8_blocks_of_larger_sizes(kind, shape):
    """Aligned operands: a layer's output, its input and weight gradients, and weights with a
    scale per row."""
    mcg = need_gpu()
    la, lb, bb = {"out": ("k_contig", "k_contig", 128), "dx": ("k_contig", "mn_contig", 128), "dw": ("mn_contig", "mn_contig", 1),
                  "rows": ("k_contig", "k_contig", 1), "mixed": ("mn_contig", "k_contig", 128)}[kind]
    M, N, K = shape
    if kind in ("dw", "mixed"):
        M = cdiv(M, 16) * 16
    for to, dtD, beta in (("e4m3", "bf16", 0.0), ("e5m2", "bf16", 0.5), ("e4m3", "f32", 1.0), ("e5m2", "f16", 0.0)):
        check_f8(mcg, to, la, lb, bb, M, N, K, dtD, 0, 0, beta)
    check_f8(mcg, "e4m3", la, lb, bb, M, N, K, "bf16", 16, 0, 0.0)


def test_gemm_f8_blocks_without_k():
    mcg = need_gpu()
    D, c = buf(6, 10, torch.float32), ref.rand(1, 6, 10).float()
    mcg.gemm_f8_blocks("e4m3", "e4m3", 0, 0, 128, 6, 10, 0, None, 1, None, 1, None, 1, None, 1, put(c), D, 10, "f32", 3.0)
    torch.cuda.synchronize()
    assert torch.equal(D.cpu(), 3 * c)


@pytest.mark.parametrize("M,N,K", [(3, 40, 300), (40, 64, 256), (300, 512, 512), (257, 256, 400)])
@pytest.mark.parametrize("dtD", ["bf16", "f32"])
def test_gemm_f8_blocks_with_scales_of_every_size(M, N, K, dtD):
    """Blocks of zeros (scale 0), scales 60 binades apart, and scales that are no numbers,
    which stay in their rows and columns."""
    mcg = need_gpu()
    qa, sa, _ = f8_operand(1, "k_contig", M, K, "e4m3", 1)
    qb, sb, _ = f8_operand(2, "k_contig", N, K, "e4m3", 128)
    sa[0] = 0.0
    sa[1, 0] *= 2.0 ** 40
    sa[1, 1:] *= 2.0 ** -40
    sb[0, -1] = 0.0
    for bad in (False, True):
        if bad:
            sa[2, 1] = float("nan")
        a, b = ref.values(qa, "e4m3", sa, 1, BLOCK), ref.values(qb, "e4m3", sb, BLOCK, BLOCK)
        A, B, SA, SB, D = put(qa), put(qb), put(sa), put(sb), buf(M, N, DT[dtD])
        mcg.gemm_f8_blocks("e4m3", "e4m3", 0, 0, 128, M, N, K, A, K, SA, ld(SA), B, K, SB, ld(SB), None, D, N, dtD)
        torch.cuda.synchronize()
        D = D.cpu()
        if bad:
            assert bool(torch.isnan(D[2]).all())
            D[2], a[2] = 0.0, 0.0
        assert not bool(D[0].any())
        d, mag = a @ b.T, a.abs() @ b.abs().T
        within(D, d, ref.tol_f8(d, mag, K, dtD), "scales")


# -------------------------------------------------------------- grouped f8
def check_grouped8(mcg, to, lb, dtD, sizes, N, K, pad=0, first=0, lead=0, tail=0):
    M, G = lead + sum(sizes) + tail, len(sizes)
    qa, sa = ref.random_codes(M + 3, M, K, to, 1, BLOCK)
    qa[:lead], qa[M - tail:] = 0x7F, 0x7F  # NaN codes
    r, c = (N, K) if lb == "k_contig" else (K, N)
    parts = [ref.random_codes(g * 3 + N, r, c, "e4m3", BLOCK, BLOCK, K ** -0.5) for g in range(G)]
    qb, sb = torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])
    b = torch.stack([ref.values(q, "e4m3", s, BLOCK, BLOCK) for q, s in parts])
    b = b.transpose(1, 2) if lb == "k_contig" else b
    off = ref.offsets_of(sizes, lead)
    A, SA, B, SB, D = put(qa, pad, first), put(sa, pad), put3(qb, pad, pad, first), put3(sb, pad, 1), buf(M, N, DT[dtD], pad, first)
    mcg.gemm_grouped_f8_blocks(to, "e4m3", lb, G, M, N, K, off.cuda(), A, ld(A), SA, ld(SA), B, ld(B), B.stride(0), SB, ld(SB),
                               SB.stride(0), D, ld(D), dtD)
    guards_hold(D)
    D = D.cpu()
    assert bool(torch.isnan(D[:lead]).all()) and bool(torch.isnan(D[M - tail:]).all()), "wrote rows of no group"
    d, mag = ref.grouped(ref.values(qa, to, sa, 1, BLOCK), b, off)
    inside = slice(lead, M - tail)
    within(D[inside], d[inside], ref.tol_f8(d[inside], mag[inside], K, dtD), f"{to} {lb} {dtD} {sizes} {N} x {K} pad {pad}")


@pytest.mark.parametrize("sizes", ["one", "uneven", "empty", "single", "last", "large"])
@pytest.mark.parametrize("lb", LAYOUTS)
def test_gemm_grouped_f8_blocks(lb, sizes):
    mcg = need_gpu()
    for i, (N, K) in enumerate([(64, 128), (130, 300), (200, 16), (129, 131), (300, 640), (4, 9)]):
        pad, first = [(0, 0), (5, 1), (16, 0)][i % 3]
        dtD = ("bf16", "f32", "f16")[i % 3]
        check_grouped8(mcg, "e5m2" if i == 1 else "e4m3", lb, dtD, SIZES[sizes], N, K, pad, first, lead=i, tail=4)


@pytest.mark.parametrize("lb", LAYOUTS)
@pytest.mark.parametrize("shape", [([900, 0, 1100, 250], 512, 512), ([300, 200, 290, 310, 100], 768, 640), ([10, 3, 20, 0, 17, 33], 1024, 768),
                                   ([1, 1, 2, 1], 2048, 2048), ([70, 50, 64, 128, 90, 1], 400, 1040)], ids=str)
def test_gemm_grouped_f8_blocks_of_larger_sizes(lb, shape):
    mcg = need_gpu()
    sizes, N, K = shape
    for to, dtD in (("e4m3", "bf16"), ("e5m2", "f32"), ("e4m3", "f16")):
        check_grouped8(mcg, to, lb, dtD, sizes, N, K, lead=5, tail=70)


# ------------------------------------------------------------- every form
@pytest.mark.parametrize("name", list(cases.GROUPED))
def test_every_form_of_gemm_grouped(name):
    mcg = need_gpu()
    case = cases.GROUPED[name]
    dt, dtD, lb, sizes, N, K, pad, kernel, tile = case
    G, M, lda, ldb, strideB = cases.operands_of_grouped(case)
    say(f"{name}: {dt} {dtD} {lb} {sizes} {N} x {K}")
    a, b, off = ref.rand(1, M, K).to(DT[dt]), (ref.rand(2, G, K, N) * K ** -0.5).to(DT[dt]), ref.offsets_of(sizes)
    A, B, D = put(a, pad), put3(b if lb == "mn_contig" else b.transpose(1, 2).contiguous(), pad), buf(M, N, DT[dtD], pad)
    assert (ld(A), ld(B), B.stride(0)) == (lda, ldb, strideB)
    assert mcg.grouped_path(dt, "k_contig", lb, G, M, N, K, A, lda, B, ldb, strideB, 128, dtD) == (kernel, tile)
    outs = []
    for _ in range(2):  # the same bits again
        D.fill_(float("nan"))
        mcg.gemm_grouped(dt, lb, G, M, N, K, off.cuda(), A, lda, B, ldb, strideB, D, ld(D), dtD)
        guards_hold(D)
        outs.append(D.cpu())
    assert torch.equal(outs[0], outs[1])
    d, mag = ref.grouped(a, b.double(), off)
    within(outs[0], d, ref.tol_16(d, mag, K, dtD), name)


@pytest.mark.parametrize("name", list(cases.GRAD))
def test_every_form_of_gemm_grouped_grad(name):
    mcg = need_gpu()
    dt, dtD, sizes, M, N, pad, kernel, tile = cases.GRAD[name]
    K, G = sum(sizes), len(sizes)
    say(f"{name}: {dt} {dtD} {sizes} {M} x {N}")
    a, b, off = ref.rand(1, K, M).to(DT[dt]), ref.rand(2, K, N).to(DT[dt]), ref.offsets_of(sizes)
    c = ref.rand(3, G, M, N).to(DT[dtD])
    A, B, C, D = put(a, pad), put(b, pad), put3(c, pad), put3(torch.zeros(G, M, N).to(DT[dtD]), pad)
    assert mcg.grouped_grad_path(dt, G, M, N, K, A, ld(A), B, ld(B), dtD) == (kernel, tile)
    d, mag = ref.grouped_grad(a, b, off, c, 0.5)
    mag = mag + 0.5 * c.double().abs()
    outs = []
    for _ in range(2):
        mcg.gemm_grouped_grad(dt, G, M, N, K, off.cuda(), A, ld(A), B, ld(B), C, D, ld(D), D.stride(0), dtD, 0.5)
        guards_hold(D)
        outs.append(D.cpu())
    assert torch.equal(outs[0], outs[1])
    within(outs[0], d, ref.tol_16(d, mag, max(sizes), dtD), name)


@pytest.mark.parametrize("name", list(cases.F8))
def test_every_form_of_gemm_f8_blocks(name):
    """With C, and over a group of all rows too where the product by group has the kind."""
    mcg = need_gpu()
    to, dtD, la, lb, bb, M, N, K, pad, kernel, tile = cases.F8[name]
    say(f"{name}: {to} {dtD} {la} {lb} {bb} {M} x {N} x {K}")
    qa, sa, a = f8_operand(1, la, M, K, to, 1)
    qb, sb, b = f8_operand(2, lb, N, K, "e4m3", bb, K ** -0.5)
    c = ref.rand(3, M, N).to(DT[dtD])
    A, B, SA, SB, C, D = put(qa, pad), put(qb, pad), put(sa), put(sb), put(c, pad), buf(M, N, DT[dtD], pad)
    assert mcg.grouped_path(to, la, lb, 0, M, N, K, A, ld(A), B, ld(B), 0, bb, dtD) == (kernel, tile)
    d, mag = a @ b.T, a.abs() @ b.abs().T
    outs = []
    for _ in range(2):
        mcg.gemm_f8_blocks(to, "e4m3", la, lb, bb, M, N, K, A, ld(A), SA, ld(SA), B, ld(B), SB, ld(SB), C, D, ld(D), dtD, 0.5)
        guards_hold(D)
        outs.append(D.cpu())
    assert torch.equal(outs[0], outs[1])
    dc, magc = d + 0.5 * c.double(), mag + 0.5 * c.double().abs()
    within(outs[0], dc, ref.tol_f8(dc, magc, K, dtD), name)
    if la == "k_contig" and bb == 128:
        off = torch.tensor([0, M], dtype=torch.int32, device="cuda")
        mcg.gemm_grouped_f8_blocks(to, "e4m3", lb, 1, M, N, K, off, A, ld(A), SA, ld(SA), B, ld(B), 0, SB, ld(SB), 0, D, ld(D), dtD)
        guards_hold(D)
        within(D, d, ref.tol_f8(d, mag, K, dtD), name + " by group")


def test_native_sums_cost_a_tenth_of_a_bf16_rounding():
    """What the documents say of the 8-bit instructions: the 2-norm of their error is below
    2^-12 of D's (measured in binary32 through a bf16 D's distance from the exact product)."""
    mcg = need_gpu()
    M, N, K = 256, 512, 4096
    qa, sa, a = f8_operand(1, "k_contig", M, K, "e4m3", 1)
    qb, sb, b = f8_operand(2, "k_contig", N, K, "e4m3", 128, K ** -0.5)
    D, E = buf(M, N, torch.bfloat16), buf(M, N, torch.float32)
    for out, dtD in ((D, "bf16"), (E, "f32")):
        mcg.gemm_f8_blocks("e4m3", "e4m3", 0, 0, 128, M, N, K, put(qa), K, put(sa), 32, put(qb), K, put(sb), 32, None, out, N, dtD)
    torch.cuda.synchronize()
    d = a @ b.T
    rel = lambda x: float((x - d).norm() / d.norm())
    rounded = rel(d.bfloat16().double())
    assert rel(E.cpu().double()) < 2.0 ** -20
    assert rel(D.cpu().double()) ** 2 - rounded ** 2 < (2.0 ** -12) ** 2, (rel(D.cpu().double()), rounded)


# ------------------------------------------------- offsets that are not valid
@pytest.mark.parametrize("off", [[0, 100, 50, 200], [-5, 40, 2 ** 31 - 1, 7], [300, 400, 500, 600], [200, 100, 0, -1],
                                 [-2 ** 31, 2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1]], ids=str)
def test_offsets_outside_the_operand_write_nothing_outside_it(off):
    """(The rows that such offsets give are tested on the host, test_group_tiles.py.)"""
    mcg = need_gpu()
    M, G = 200, 3
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    for N, K in ((256, 256), (40, 72), (130, 67), (3, 2)):
        a, b = ref.rand(1, M, K).bfloat16(), ref.rand(2, G, N, K).bfloat16()
        A, B, D = put(a), put3(b), buf(M, N, torch.bfloat16)
        mcg.gemm_grouped("bf16", "k_contig", G, M, N, K, o, A, K, B, K, B.stride(0), D, N, "bf16")
        guards_hold(A, B, D)
        x, y, W = put(ref.rand(3, M, K).bfloat16()), put(ref.rand(4, M, N).bfloat16()), put3(torch.zeros(G, K, N))
        mcg.gemm_grouped_grad("bf16", G, K, N, M, o, x, K, y, N, None, W, N, W.stride(0), "f32")
        guards_hold(x, y, W)
        q = torch.zeros(M, K, dtype=torch.uint8)
        A8, B8 = put(q), put3(torch.zeros(G, N, K, dtype=torch.uint8))
        SA, SB = put(torch.ones(M, cdiv(K, BLOCK))), put3(torch.ones(G, cdiv(N, BLOCK), cdiv(K, BLOCK)))
        mcg.gemm_grouped_f8_blocks("e4m3", "e4m3", "k_contig", G, M, N, K, o, A8, K, SA, ld(SA), B8, K, B8.stride(0), SB, ld(SB),
                                   SB.stride(0), D, N, "bf16")
        guards_hold(A8, B8, D)


# ----------------------------------------------------- a run of them together
def expert_state(T, K, N, sizes):
    """Buffers of an expert layer y = W_g x: rows sorted by expert."""
    bf = torch.bfloat16
    G = len(sizes)
    w = (ref.rand(7, G, N, K) * K ** -0.5).to(bf)
    f = lambda *s: torch.full(s, float("nan"), device="cuda")
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")
    return {"x": put(ref.rand(1, T, K).to(bf)), "w": w.cuda(), "dy": put(ref.rand(2, T, N).to(bf)), "off": ref.offsets_of(sizes).cuda(),
            "y": f(T, N).to(bf), "y8": f(T, N).to(bf), "dx": f(T, K).to(bf), "dw": f(G, N, K), "qx": u8(T, K), "sx": f(T, cdiv(K, BLOCK)),
            "qw": u8(G, N, K), "sw": f(G, cdiv(N, BLOCK), cdiv(K, BLOCK)), "xb": f(T, K).to(bf)}


def expert_step(mcg, s, T, K, N, G, stream=None):
    """Forward in 16 bits and in 8, backward in 16."""
    KB, NB = cdiv(K, BLOCK), cdiv(N, BLOCK)
    mcg.gemm_grouped("bf16", "k_contig", G, T, N, K, s["off"], s["x"], K, s["w"], K, N * K, s["y"], N, "bf16", stream)
    for g in range(G):
        mcg.quantize_blocks("bf16", "e4m3", 128, 128, N, K, s["w"][g], K, s["qw"][g], K, s["sw"][g], KB, stream)
    mcg.quantize_blocks("bf16", "e4m3", 1, 128, T, K, s["x"], K, s["qx"], K, s["sx"], KB, stream)
    mcg.gemm_grouped_f8_blocks("e4m3", "e4m3", "k_contig", G, T, N, K, s["off"], s["qx"], K, s["sx"], KB, s["qw"], K, N * K, s["sw"], KB,
                               NB * KB, s["y8"], N, "bf16", stream)
    mcg.dequantize_blocks("e4m3", "bf16", 1, 128, T, K, s["qx"], K, s["sx"], KB, s["xb"], K, stream)
    mcg.gemm_grouped("bf16", "mn_contig", G, T, K, N, s["off"], s["dy"], N, s["w"], K, N * K, s["dx"], K, "bf16", stream)
    mcg.gemm_grouped_grad("bf16", G, N, K, T, s["off"], s["dy"], N, s["xb"], K, None, s["dw"], K, N * K, "f32", 0.0, stream)


OUTS = ("y", "y8", "dx", "dw", "qx", "sx", "qw", "sw", "xb")
STEPS = [(64, 48, [3, 0, 2]), (256, 384, [100, 1, 0, 260, 63]), (130, 70, [40, 9]), (512, 256, [2, 1, 0, 1, 4])]


@pytest.mark.parametrize("K,N,sizes", STEPS, ids=str)
def test_an_expert_layers_step(K, N, sizes):
    """Against the formulas; the gradients against differences of the forward product too."""
    mcg = need_gpu()
    T, G = sum(sizes), len(sizes)
    s = expert_state(T, K, N, sizes)
    expert_step(mcg, s, T, K, N, G)
    torch.cuda.synchronize()
    off, x, w, dy = s["off"].cpu(), s["x"].cpu(), s["w"].cpu().double(), s["dy"].cpu()
    y, mag = ref.grouped(x, w.transpose(1, 2), off)
    within(s["y"], y, ref.tol_16(y, mag, K, "bf16"), "y")
    dx, mag = ref.grouped(dy, w, off)
    within(s["dx"], dx, ref.tol_16(dx, mag, N, "bf16"), "dx")
    xq = ref.values(s["qx"].cpu(), "e4m3", s["sx"].cpu(), 1, BLOCK)
    wq = torch.stack([ref.values(s["qw"][g].cpu(), "e4m3", s["sw"][g].cpu(), BLOCK, BLOCK) for g in range(G)])
    y8, mag8 = ref.grouped(xq, wq.transpose(1, 2), off)
    within(s["y8"], y8, ref.tol_f8(y8, mag8, K, "bf16"), "y8")
    xb = s["xb"].cpu()
    within(xb, xq, (ref.U["bf16"] + 2 * ref.U32) * xq.abs() + ref.SUB["bf16"], "xb")
    dw, magw = ref.grouped_grad(dy, xb, off, None, 0.0)
    within(s["dw"], dw, ref.tol_16(dw, magw, T, "f32"), "dw")
    # f(W, X) = sum of dy * y is linear: a step along a direction changes it by the gradient's product with it
    r = np.random.default_rng(0)
    V, U_ = torch.from_numpy(r.standard_normal(tuple(w.shape))), torch.from_numpy(r.standard_normal((T, K)))
    f = lambda W, X: float((dy.double() * torch.nan_to_num(ref.grouped(X, W.transpose(1, 2), off)[0])).sum())
    diff_w, diff_x = (f(w + V, xb.double()) - f(w - V, xb.double())) / 2, (f(w, x.double() + U_) - f(w, x.double() - U_)) / 2
    got_w, got_x = float((s["dw"].cpu().double() * V).sum()), float((s["dx"].cpu().double() * U_).sum())
    # (each gradient within its tolerance, so its product with the direction is)
    assert abs(got_w - diff_w) <= float((ref.tol_16(dw, magw, T, "f32") * V.abs()).sum()) + 1e-9 * float((magw * V.abs()).sum())
    assert abs(got_x - diff_x) <= float((ref.tol_16(dx, mag, N, "bf16") * U_.abs()).sum()) + 1e-9 * float((mag * U_.abs()).sum())


@pytest.mark.parametrize("K,N,sizes", STEPS, ids=str)
def test_an_expert_layers_step_on_another_stream_and_in_a_graph(K, N, sizes):
    """The same bits eagerly, on another stream beside other work, and replayed; a replay
    follows offsets that changed since the capture."""
    mcg = need_gpu()
    T, G = sum(sizes), len(sizes)
    s = expert_state(T, K, N, sizes)
    other = expert_state(T, K, N, sizes)

    def reset(t):
        for k in OUTS:
            t[k].fill_(0x33 if t[k].dtype == torch.uint8 else float("nan"))
        torch.cuda.synchronize()

    def same(expect, what):
        torch.cuda.synchronize()
        for k in OUTS:
            assert torch.equal(s[k].view(torch.uint8), expect[k].view(torch.uint8)), f"{what}: {k}"

    def eager_of():
        reset(s)
        expert_step(mcg, s, T, K, N, G)
        torch.cuda.synchronize()
        return {k: s[k].clone() for k in OUTS}
    eager = eager_of()
    st, st2 = torch.cuda.Stream(), torch.cuda.Stream()
    reset(s)
    expert_step(mcg, s, T, K, N, G, st)
    expert_step(mcg, other, T, K, N, G, st2)  # at the same time
    same(eager, "another stream")
    for k in OUTS:
        assert torch.equal(other[k].view(torch.uint8), eager[k].view(torch.uint8)), k
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        expert_step(mcg, s, T, K, N, G, st)
    for rep in range(3):
        reset(s)
        g.replay()
        same(eager, f"replay {rep}")
    s["off"].copy_(ref.offsets_of(list(reversed(sizes))))
    changed = eager_of()
    reset(s)
    g.replay()
    same(changed, "replay with other offsets")
    say(f"  {K} x {N} {sizes}: same bits on other streams and in replays")


# --------------------------------------------------------------------- the example
def test_the_example_runs_and_its_gradients_hold():
    """Gradients against the formulas over the tensors that the layer quantised, and against
    differences of the forward product."""
    need_gpu()
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_layer.py")
    spec = importlib.util.spec_from_file_location("expert_layer", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    T, K, N, G = 200, 192, 256, 5
    layer = example.ExpertLayer(T, K, N, G)
    x, dy = ref.rand(1, T, K).bfloat16().cuda(), ref.rand(2, T, N).bfloat16().cuda()
    expert = torch.from_numpy(np.random.default_rng(3).integers(0, G - 1, T)).cuda()  # (one expert has no token)
    y, dx = layer.forward(x, expert), layer.backward(dy)
    torch.cuda.synchronize()
    order, off = layer.order.cpu(), layer.offsets.cpu()
    val = lambda q, to, s, bm, bn: ref.values(q.cpu(), to, s.cpu(), bm, bn)
    w = torch.stack([val(layer.qw[g], "e4m3", layer.sw[g], BLOCK, BLOCK) for g in range(G)])
    ws = val(layer.qws, "e4m3", layer.sws, BLOCK, BLOCK)
    xq, dyq = val(layer.qx, "e4m3", layer.sx, 1, BLOCK), val(layer.qdy, "e5m2", layer.sdy, 1, BLOCK)
    xt, dyt = val(layer.qxt, "e4m3", layer.sxt, BLOCK, 1), val(layer.qdyt, "e5m2", layer.sdyt, BLOCK, 1)

    def two(a, b, bs, k):  # the experts' product, rounded, is the C of the shared one
        d, mag = ref.grouped(a, b, off)
        tol = ref.tol_f8(d, mag, k, "bf16")
        return d + a @ bs, tol + ref.tol_f8(d + a @ bs, mag + a.abs() @ bs.abs(), k, "bf16") + 2 * ref.U["bf16"] * tol
    exact, tol = two(xq, w.transpose(1, 2), ws.T, K)
    within(y.cpu()[order], exact, tol, "y")
    dx_exact, dx_tol = two(dyq, w, ws, N)
    within(dx.cpu()[order], dx_exact, dx_tol, "dx")
    dw, mag = ref.grouped_grad(layer.dy.cpu(), layer.x.cpu(), off, None, 0.0)
    dw_tol = ref.tol_16(dw, mag, T, "f32")
    within(layer.dw, dw, dw_tol, "dw")
    dws, mags = dyt.T @ xt, dyt.abs().T @ xt.abs()
    dws_tol = ref.tol_f8(dws, mags, T, "f32")
    within(layer.dws, dws, dws_tol, "dws")
    # sum of dy * y is linear in each of x, w and ws: a step along a direction changes it by the gradient's
    # product with the direction
    r = np.random.default_rng(4)
    f = lambda X, W, WS, DY: float((DY * (ref.grouped(X, W.transpose(1, 2), off)[0] + X @ WS.T)).sum())
    V = torch.from_numpy(r.standard_normal((T, K)))
    change = (f(xq + V, w, ws, dyq) - f(xq - V, w, ws, dyq)) / 2
    assert abs(float((dx.cpu()[order].double() * V).sum()) - change) <= float((dx_tol * V.abs()).sum()) * (1 + 1e-9)
    V, xb, dyb = torch.from_numpy(r.standard_normal((G, N, K))), layer.x.cpu().double(), layer.dy.cpu().double()
    change = (f(xb, w + V, ws, dyb) - f(xb, w - V, ws, dyb)) / 2
    assert abs(float((layer.dw.cpu().double() * V).sum()) - change) <= float((dw_tol * V.abs()).sum()) * (1 + 1e-9)
    V = torch.from_numpy(r.standard_normal((N, K)))
    change = (f(xt, w, ws + V, dyt) - f(xt, w, ws - V, dyt)) / 2
    assert abs(float((layer.dws.cpu().double() * V).sum()) - change) <= float((dws_tol * V.abs()).sum()) * (1 + 1e-9)
    assert len(example.train(T=100, K=128, N=128, G=3, steps=2)) == 2
