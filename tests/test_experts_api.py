"""Argument checks of the products by group and of block-scaled 8-bit floats: every
refusal is found on the host, before any HIP call, so no GPU is needed; the binding
with and without its C extension; and the plain forms of the GPU tests."""
import ctypes

import pytest
import torch

import experts_ref as ref

m = pytest.importorskip("matrix_core_gemm_amd")

FAKE = 0x10000  # aligned and non-null; never dereferenced here


def check(validate, base, kw, status):
    a = dict(base)
    a.update(kw)
    assert validate(**a) == status


QUANT = dict(dtype="bf16", dtypeQ="e4m3", blockM=1, blockN=128, M=4, N=300, X=FAKE, ldx=300, Q=FAKE, ldq=300, scale=FAKE, lds=3)


@pytest.mark.parametrize("kw,status", [
    ({}, 0), ({"dtype": "f16"}, 0), ({"dtype": "f32"}, 0), ({"dtypeQ": "e5m2"}, 0),
    ({"dtype": "i8"}, 4), ({"dtypeQ": "i8"}, 4), ({"dtypeQ": "bf16"}, 4), ({"dtype": 42}, 4),
    ({"blockN": 64}, 10), ({"blockM": 128, "blockN": 1, "lds": 300}, 0), ({"blockM": 128, "blockN": 128}, 0),
    ({"blockN": 1}, 10), ({"blockM": 2}, 10), ({"blockM": 0}, 10), ({"blockM": -1}, 10),
    ({"M": -1}, 2), ({"N": 1 << 31}, 2), ({"M": 0, "X": None, "Q": None, "scale": None}, 0), ({"N": 0, "X": None}, 0),
    ({"X": None}, 1), ({"Q": None}, 1), ({"scale": None}, 1),
    ({"ldx": 299}, 3), ({"ldq": 299}, 3), ({"lds": 2}, 3), ({"blockM": 128, "blockN": 1, "lds": 299}, 3),
    ({"X": FAKE + 1}, 5), ({"scale": FAKE + 2}, 5), ({"Q": FAKE + 1}, 0), ({"X": FAKE + 2, "ldx": 301}, 0),
    ({"dtype": "f32", "X": FAKE + 2}, 5),
])
def test_quantize_blocks_validation(kw, status):
    check(m.validate_quantize_blocks, QUANT, kw, status)
    if not set(kw) & {"dtype", "X", "ldx"}:
        back = {"dtypeQ": "e4m3", "dtypeD": "bf16", "blockM": 1, "blockN": 128, "M": 4, "N": 300, "Q": FAKE, "ldq": 300,
                "scale": FAKE, "lds": 3, "D": FAKE, "ldd": 300}
        check(m.validate_dequantize_blocks, back, kw, status)


@pytest.mark.parametrize("kw,status", [
    ({"dtypeD": "i8"}, 4), ({"D": None}, 1), ({"ldd": 299}, 3), ({"D": FAKE + 1}, 5), ({"dtypeD": "f32", "D": FAKE + 2}, 5),
])
def test_dequantize_blocks_validation(kw, status):
    check(m.validate_dequantize_blocks, dict(dtypeQ="e5m2", dtypeD="f16", blockM=128, blockN=128, M=4, N=300, Q=FAKE, ldq=300,
                                             scale=FAKE, lds=3, D=FAKE, ldd=300), kw, status)


F8 = dict(dtypeA="e4m3", dtypeB="e4m3", layoutA="k_contig", layoutB="k_contig", blockB=128, M=8, N=200, K=300, A=FAKE, lda=300,
          scaleA=FAKE, ldsa=3, B=FAKE, ldb=300, scaleB=FAKE, ldsb=3, C=None, D=FAKE, ldd=200, dtypeD="bf16", beta=0.0)


@pytest.mark.parametrize("kw,status", [
    ({}, 0), ({"dtypeA": "e5m2"}, 0), ({"dtypeB": "e5m2"}, 4), ({"dtypeA": "bf16"}, 4), ({"dtypeD": "i32"}, 4),
    ({"dtypeD": "f16"}, 0), ({"dtypeD": "f32"}, 0), ({"layoutA": 2}, 4), ({"layoutB": -1}, 4),
    ({"blockB": 1}, 0), ({"blockB": 64}, 10), ({"blockB": 0}, 10), ({"beta": float("nan")}, 10), ({"beta": 1e39, "C": FAKE}, 10),
    ({"beta": 1.0}, 1), ({"beta": 1.0, "C": FAKE}, 0), ({"beta": 1.0, "C": FAKE + 1}, 5),
    ({"M": -1}, 2), ({"K": 1 << 31}, 2), ({"M": 0, "A": None, "D": None}, 0), ({"N": 0}, 0),
    ({"K": 0, "A": None, "B": None, "scaleA": None, "scaleB": None, "lda": 1, "ldb": 1, "ldsa": 1, "ldsb": 1}, 0),
    ({"A": None}, 1), ({"B": None}, 1), ({"scaleA": None}, 1), ({"scaleB": None}, 1), ({"D": None}, 1),
    ({"lda": 299}, 3), ({"ldb": 299}, 3), ({"ldd": 199}, 3), ({"ldsa": 2}, 3), ({"ldsb": 2}, 3),
    ({"layoutA": "mn_contig", "lda": 8, "ldsa": 8}, 0), ({"layoutA": "mn_contig", "lda": 7, "ldsa": 8}, 3),
    ({"layoutA": "mn_contig", "lda": 8, "ldsa": 7}, 3),
    ({"layoutB": "mn_contig", "ldb": 200, "ldsb": 2}, 0), ({"layoutB": "mn_contig", "ldb": 200, "ldsb": 1}, 3),
    ({"layoutB": "mn_contig", "blockB": 1, "ldb": 200, "ldsb": 199}, 3),
    ({"layoutB": "mn_contig", "blockB": 1, "ldb": 200, "ldsb": 200}, 0),
    ({"scaleA": FAKE + 1}, 5), ({"scaleB": FAKE + 2}, 5), ({"A": FAKE + 1, "B": FAKE + 3}, 0), ({"D": FAKE + 1}, 5),
])
def test_f8_blocks_validation(kw, status):
    check(m.validate_f8_blocks, F8, kw, status)


GROUPED = dict(dtype="bf16", layoutB="k_contig", G=3, M=8, N=40, K=64, offsets=FAKE, A=FAKE, lda=64, B=FAKE, ldb=64,
               strideB=40 * 64, D=FAKE, ldd=40, dtypeD="bf16")


@pytest.mark.parametrize("kw,status", [
    ({}, 0), ({"dtype": "f16"}, 4), ({"dtype": "f16", "dtypeD": "f16"}, 0), ({"dtypeD": "f32"}, 0), ({"dtype": "f32"}, 4),
    ({"dtype": "e4m3", "dtypeD": "f32"}, 4), ({"layoutB": 3}, 4), ({"G": -1}, 2), ({"G": 65536}, 2), ({"G": 65535}, 0),
    ({"G": 0, "offsets": None, "D": None}, 0), ({"M": 0, "A": None, "D": None}, 0), ({"N": 0}, 0), ({"strideB": -1}, 2),
    ({"strideB": 0}, 0), ({"M": 1 << 31}, 2), ({"offsets": None}, 1), ({"A": None}, 1), ({"B": None}, 1), ({"D": None}, 1),
    ({"K": 0, "A": None, "B": None, "lda": 1, "ldb": 1}, 0), ({"lda": 63}, 3), ({"ldb": 63}, 3), ({"ldd": 39}, 3),
    ({"layoutB": "mn_contig", "ldb": 39}, 3), ({"layoutB": "mn_contig", "ldb": 40}, 0),
    ({"offsets": FAKE + 2}, 5), ({"A": FAKE + 1}, 5), ({"B": FAKE + 1}, 5), ({"A": FAKE + 2}, 0), ({"dtypeD": "f32", "D": FAKE + 2}, 5),
])
def test_grouped_validation(kw, status):
    check(m.validate_grouped, GROUPED, kw, status)


GRAD = dict(dtype="bf16", G=3, M=8, N=40, K=64, offsets=FAKE, A=FAKE, lda=8, B=FAKE, ldb=40, C=None, D=FAKE, ldd=40, strideD=320,
            dtypeD="f32", beta=0.0)


@pytest.mark.parametrize("kw,status", [
    ({}, 0), ({"dtype": "e4m3"}, 4), ({"dtypeD": "f16"}, 4), ({"G": 65536}, 2), ({"K": -1}, 2), ({"G": 0, "D": None}, 0),
    ({"beta": 1.0}, 1), ({"beta": 1.0, "C": FAKE}, 0), ({"beta": float("inf"), "C": FAKE}, 10), ({"offsets": None}, 1), ({"A": None}, 1),
    ({"K": 0, "offsets": None, "A": None, "B": None}, 0), ({"D": None}, 1), ({"lda": 7}, 3), ({"ldb": 39}, 3), ({"ldd": 39}, 3),
    ({"strideD": 319}, 3), ({"strideD": 0, "G": 1}, 0), ({"ldd": 41, "strideD": 7 * 41 + 39}, 3), ({"ldd": 41, "strideD": 7 * 41 + 40}, 0),
    ({"offsets": FAKE + 1}, 5), ({"A": FAKE + 1}, 5), ({"D": FAKE + 2}, 5), ({"beta": 1.0, "C": FAKE + 2}, 5), ({"M": 0}, 0),
])
def test_grouped_grad_validation(kw, status):
    check(m.validate_grouped_grad, GRAD, kw, status)


GROUPED8 = dict(dtypeA="e4m3", dtypeB="e4m3", layoutB="k_contig", G=3, M=8, N=200, K=300, offsets=FAKE, A=FAKE, lda=300, scaleA=FAKE,
                ldsa=3, B=FAKE, ldb=300, strideB=60000, scaleB=FAKE, ldsb=3, strideSB=6, D=FAKE, ldd=200, dtypeD="bf16")


@pytest.mark.parametrize("kw,status", [
    ({}, 0), ({"dtypeA": "e5m2"}, 0), ({"dtypeB": "e5m2"}, 4), ({"dtypeD": "i8"}, 4), ({"G": 65536}, 2), ({"strideSB": -1}, 2),
    ({"offsets": None}, 1), ({"scaleA": None}, 1), ({"scaleB": None}, 1), ({"ldsa": 2}, 3), ({"ldsb": 2}, 3),
    ({"layoutB": "mn_contig", "ldb": 200, "ldsb": 2}, 0), ({"layoutB": "mn_contig", "ldb": 200, "ldsb": 1}, 3),
    ({"scaleB": FAKE + 2}, 5), ({"G": 0, "D": None}, 0), ({"M": 0}, 0), ({"strideB": 0, "strideSB": 0}, 0),
])
def test_grouped_f8_blocks_validation(kw, status):
    check(m.validate_grouped_f8_blocks, GROUPED8, kw, status)


CALLS = [("quantize_blocks", QUANT), ("dequantize_blocks", dict(dtypeQ="e5m2", dtypeD="f16", blockM=128, blockN=128, M=4, N=300,
                                                                 Q=FAKE, ldq=300, scale=FAKE, lds=3, D=FAKE, ldd=300)),
         ("gemm_f8_blocks", F8), ("gemm_grouped", GROUPED), ("gemm_grouped_grad", GRAD), ("gemm_grouped_f8_blocks", GROUPED8)]


@pytest.mark.parametrize("name,base", CALLS, ids=[c[0] for c in CALLS])
def test_entry_points_reject_before_touching_the_device(name, base):
    """The same refusals from the entry point, by the C extension and by ctypes."""
    for change, status in (({"D" if "D" in base else "Q": None}, 1), ({"M": -1}, 2), ({"M": 1 << 31}, 2)):
        a = {**base, **change}
        with pytest.raises(m.MCGError) as e:
            getattr(m, name)(**a, stream=0)
        assert e.value.status == status
        positional = list(a.values()) + [0]
        assert getattr(m._mcgcall, name)(*positional) == status
        assert getattr(m._CtypesCalls(), name)(*positional) == status
    for side in (m._mcgcall, m._CtypesCalls()):
        positional = list({**base, "M": -1}.values()) + [0]
        for bad, error in ((positional[:-1], TypeError), (["no type"] + positional[1:], KeyError),
                           ([p if k != "M" else 1 << 70 for k, p in zip([*base, "stream"], positional)], OverflowError),
                           ([p if k != "M" else 1.5 for k, p in zip([*base, "stream"], positional)], TypeError)):
            with pytest.raises(error):
                getattr(side, name)(*bad)
    getattr(m, name)(**{**base, "M": 0}, stream=0)  # an empty product is no call of the device


@pytest.mark.parametrize("side", ["extension", "ctypes"])
def test_no_long_integer_wraps_into_a_block(side):
    call = m._mcgcall if side == "extension" else m._CtypesCalls()
    a = list({**QUANT, "blockN": (1 << 32) + 128}.values()) + [0]
    assert call.quantize_blocks(*a) == 10
    a = list({**F8, "blockB": (1 << 32) + 1}.values()) + [0]
    assert call.gemm_f8_blocks(*a) == 10


def test_path_queries_refuse_what_the_calls_refuse():
    assert m.grouped_path("f32", 0, 0, 2, 4, 64, 64, FAKE, 64, FAKE, 64, 0, 128, "f32")[0] == -1
    assert m.grouped_path("bf16", 0, 0, 2, 0, 64, 64, FAKE, 64, FAKE, 64, 0, 128, "bf16")[0] == -1
    assert m.grouped_grad_path("bf16", 0, 4, 64, 64, FAKE, 64, FAKE, 64, "bf16")[0] == -1
    assert m.grouped_path("bf16", 0, 0, 2, 1, 64, 3, FAKE, 64, FAKE, 64, 0, 128, "bf16")[0] == 16
    assert m.grouped_grad_path("bf16", 2, 4, 64, 64, FAKE, 64, FAKE, 64, "bf16")[0] == 16
    assert m.lib().mcg_grouped_path(0, 0, 0, 2, 4, 64, 64, FAKE, 64, FAKE, 64, 0, 128, 0, ctypes.c_void_p(0)) >= 0


# ------------------------------------------------------------------- the plain forms
@pytest.mark.parametrize("to", ["e4m3", "e5m2"])
@pytest.mark.parametrize("kind", list(ref.KINDS))
def test_plain_quantize_is_off_by_half_a_step(to, kind):
    bm, bn = ref.KINDS[kind]
    x = ref.rand(3, 150, 300).bfloat16().float()
    x[:, 17] *= 40
    q, scale = ref.quantize(x, to, bm, bn)
    v = ref.values(q, to, scale, bm, bn)
    s = ref.per_element(scale.double(), 150, 300, bm, bn)
    half, low = (2.0 ** -4, 2.0 ** -9) if to == "e4m3" else (2.0 ** -3, 2.0 ** -16)
    assert bool(((v - x.double()).abs() <= half * x.double().abs() * (1 + 2.0 ** -20) + low / 2 * s + 2.0 ** -23 * x.double().abs()).all())
    assert int((q.view(ref.F8[to]).float().abs() == ref.LARGEST[to]).sum()) >= scale.numel()


def test_plain_products_agree_with_loops():
    a, b = ref.rand(1, 9, 5), ref.rand(2, 3, 5, 4)
    off = ref.offsets_of([2, 0, 4], first=1)
    d, mag = ref.grouped(a, b, off)
    assert torch.isnan(d[0]).all() and torch.isnan(d[7:]).all()
    assert torch.allclose(d[1], a[1] @ b[0]) and torch.allclose(d[6], a[6] @ b[2]) and bool((mag[1:7] >= d[1:7].abs()).all())
    x, y = ref.rand(3, 9, 2), ref.rand(4, 9, 6)
    g, _ = ref.grouped_grad(x, y, off, None, 0.0)
    assert torch.allclose(g[0], sum(x[r][:, None] * y[r] for r in (1, 2))) and not g[1].any()


@pytest.mark.parametrize("validate,base,fits,not_fit", [
    (m.validate_quantize_blocks, QUANT, dict(M=1, N=128 * (2**24 - 1)), dict(M=1, N=128 * (2**24 - 1) + 1)),
    (m.validate_f8_blocks, F8, dict(M=64 * 4096, N=128 * 2047), dict(M=64 * 4096, N=128 * 2048)),
    (m.validate_grouped, GROUPED, dict(G=65535, M=65535, N=128 * 127), dict(G=65535, M=65535, N=128 * 128 + 1)),
    (m.validate_grouped_grad, GRAD, dict(G=65535, M=128, N=128 * 127), dict(G=65535, M=129, N=128 * 64 + 1)),
    (m.validate_grouped_f8_blocks, GROUPED8, dict(G=65535, M=65535 * 64, N=128 * 64), dict(G=65535, M=65535 * 64, N=128 * 65)),
], ids=["quantize_blocks", "f8_blocks", "grouped", "grouped_grad", "grouped_f8_blocks"])
def test_more_tiles_than_a_launch_holds_are_refused(validate, base, fits, not_fit):
    big = 1 << 40  # leading dimensions and strides of any size
    for sizes, status in ((fits, 0), (not_fit, 2)):
        lds = {k: big for k in base if k.startswith("ld")}
        if "strideD" in base:
            lds["strideD"] = 1 << 60
        check(validate, base, {**lds, **sizes}, status)
