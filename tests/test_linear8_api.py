"""Argument checks of the 8-bit linear layer's entry points: every refusal is
found on the host, before any HIP call, so no GPU is needed."""
import ctypes

import pytest

m = pytest.importorskip("matrix_core_gemm_amd")

FAKE = 0x10000  # aligned and non-null; never dereferenced here
BIG = 1 << 40


def rmsnorm_quant_args(**kw):
    a = dict(dtype="bf16", M=4, N=64, X=FAKE, ldx=64, R=FAKE, ldr=64, weight=FAKE, eps=1e-5, H=FAKE, ldh=64, Q=FAKE,
             ldq=64, scale=FAKE, rstd=FAKE)
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,status", [
    ({}, 0),
    ({"dtype": "f16"}, 0), ({"dtype": "f32"}, 0),
    ({"dtype": "i8"}, 4), ({"dtype": "f64"}, 4), ({"dtype": "e4m3"}, 4), ({"dtype": 42}, 4),
    ({"M": -1}, 2), ({"N": -1}, 2), ({"M": 1 << 31}, 2), ({"N": 1 << 31}, 2),
    ({"eps": -1e-6}, 10), ({"eps": float("nan")}, 10), ({"eps": float("inf")}, 10), ({"eps": 1e39}, 10),
    ({"eps": 0.0}, 0),
    ({"M": 0, "X": None, "Q": None, "scale": None}, 0),
    ({"X": None}, 1), ({"Q": None}, 1), ({"scale": None}, 1),
    ({"N": 0, "X": None, "Q": None}, 0), ({"N": 0, "scale": None}, 1),
    ({"R": None, "ldr": 0, "weight": None, "H": None, "ldh": 0, "rstd": None}, 0),
    ({"ldx": 63}, 3), ({"ldr": 63}, 3), ({"ldh": 63}, 3), ({"ldq": 63}, 3),
    ({"X": FAKE + 1}, 5), ({"R": FAKE + 1}, 5), ({"weight": FAKE + 1}, 5), ({"H": FAKE + 1}, 5),
    ({"Q": FAKE + 1}, 0), ({"scale": FAKE + 2}, 5), ({"rstd": FAKE + 2}, 5),
    ({"X": FAKE + 2, "ldx": 65, "Q": FAKE + 3, "ldq": 67}, 0),  # any element alignment
    ({"dtype": "f32", "X": FAKE + 2}, 5),
])
def test_rmsnorm_quant_validation(kw, status):
    assert m.validate_rmsnorm_quant(**rmsnorm_quant_args(**kw)) == status


def rmsnorm_backward_args(**kw):
    a = dict(dtype="bf16", dtypeX="bf16", M=4, N=64, dY=FAKE, lddy=64, X=FAKE, ldx=64, scaleX=None, weight=FAKE,
             rstd=FAKE, dR=FAKE, lddr=64, dX=FAKE, lddx=64, dW=FAKE, workspace=FAKE, workspace_bytes=BIG)
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,status", [
    ({}, 0),
    ({"dtype": "i8", "dtypeX": "i8"}, 4), ({"dtypeX": "f16"}, 4), ({"dtypeX": "f32"}, 4),
    ({"dtypeX": "i8"}, 1), ({"dtypeX": "i8", "scaleX": FAKE}, 0), ({"dtypeX": "i8", "scaleX": FAKE, "X": FAKE + 1}, 0),
    ({"dtypeX": "i8", "scaleX": FAKE + 1}, 5),
    ({"M": -1}, 2), ({"N": 1 << 31}, 2), ({"workspace_bytes": -1}, 2),
    ({"N": 0, "dY": None}, 0),
    ({"dY": None}, 1), ({"X": None}, 1), ({"rstd": None}, 1), ({"dX": None}, 1),
    ({"M": 0, "dY": None, "X": None, "rstd": None, "dX": None, "workspace": None, "workspace_bytes": 0}, 0),
    ({"dR": None, "lddr": 0, "weight": None}, 0),
    ({"lddy": 63}, 3), ({"ldx": 63}, 3), ({"lddr": 63}, 3), ({"lddx": 63}, 3),
    ({"dY": FAKE + 1}, 5), ({"X": FAKE + 1}, 5), ({"dR": FAKE + 1}, 5), ({"dX": FAKE + 1}, 5), ({"dW": FAKE + 2}, 5),
    ({"workspace": FAKE + 8}, 5),
    ({"workspace": None}, 11), ({"workspace_bytes": 4 * 64 * 4 - 1}, 11), ({"workspace_bytes": 4 * 64 * 4}, 0),
    ({"dW": None, "workspace": None, "workspace_bytes": 0}, 0),
])
def test_rmsnorm_backward_validation(kw, status):
    assert m.validate_rmsnorm_backward(**rmsnorm_backward_args(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    ({}, 0), ({"dtype": "f32"}, 0), ({"dtype": "i8"}, 4), ({"M": -1}, 2), ({"N": 1 << 31}, 2),
    ({"M": 0, "X": None, "Q": None, "scale": None}, 0), ({"X": None}, 1), ({"Q": None}, 1), ({"scale": None}, 1),
    ({"ldx": 63}, 3), ({"ldq": 63}, 3), ({"X": FAKE + 1}, 5), ({"scale": FAKE + 1}, 5), ({"Q": FAKE + 1}, 0),
])
def test_quantize_rows_validation(kw, status):
    a = dict(dtype="bf16", M=4, N=64, X=FAKE, ldx=64, Q=FAKE, ldq=64, scale=FAKE)
    a.update(kw)
    assert m.validate_quantize_rows(**a) == status


@pytest.mark.parametrize("kw,status", [
    ({}, 0), ({"dtypeD": "f16"}, 0), ({"dtypeD": "i32"}, 4), ({"M": -1}, 2), ({"N": 1 << 31}, 2),
    ({"M": 0, "Q": None, "scale": None, "D": None}, 0), ({"N": 0, "Q": None, "scale": None, "D": None}, 0),
    ({"Q": None}, 1), ({"scale": None}, 1), ({"D": None}, 1), ({"ldq": 63}, 3), ({"ldd": 63}, 3),
    ({"D": FAKE + 1}, 5), ({"scale": FAKE + 2}, 5), ({"Q": FAKE + 1, "ldq": 65}, 0),
])
def test_dequantize_rows_validation(kw, status):
    a = dict(dtypeD="bf16", M=4, N=64, Q=FAKE, ldq=64, scale=FAKE, D=FAKE, ldd=64)
    a.update(kw)
    assert m.validate_dequantize_rows(**a) == status


def i8_scaled_args(**kw):
    a = dict(layoutB="k_contig", M=8, N=32, K=48, A=FAKE, lda=48, scaleA=FAKE, B=FAKE, ldb=48, scaleB=FAKE, bias=None,
             D=FAKE, ldd=32, dtypeD="bf16", workspace=None, workspace_bytes=0)
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,status", [
    ({}, 0), ({"dtypeD": "f32"}, 0), ({"dtypeD": "f16", "bias": FAKE}, 0),
    ({"dtypeD": "i32"}, 4), ({"dtypeD": "i8"}, 4), ({"layoutB": 2}, 4),
    ({"M": -1}, 2), ({"N": -1}, 2), ({"K": -1}, 2), ({"M": 1 << 31}, 2),
    ({"K": 131071, "lda": 131071, "ldb": 131071}, 0), ({"K": 131072, "lda": 131072, "ldb": 131072}, 2),
    ({"M": 0, "A": None, "D": None}, 0), ({"N": 0, "ldd": 0, "D": None}, 0),
    ({"A": None}, 1), ({"B": None}, 1), ({"D": None}, 1), ({"scaleA": None}, 1), ({"scaleB": None}, 1),
    ({"K": 0, "A": None, "B": None, "lda": 1, "ldb": 1}, 0),
    ({"lda": 47}, 3), ({"ldb": 47}, 3), ({"ldd": 31}, 3),
    ({"layoutB": "mn_contig", "ldb": 31}, 3), ({"layoutB": "mn_contig", "ldb": 32}, 0),
    ({"scaleA": FAKE + 2}, 5), ({"scaleB": FAKE + 1}, 5), ({"bias": FAKE + 2}, 5), ({"D": FAKE + 1}, 5),
    ({"A": FAKE + 1, "B": FAKE + 3, "D": FAKE + 2}, 0),
    ({"workspace": FAKE + 4, "workspace_bytes": 64}, 5), ({"workspace_bytes": -1}, 2),
    ({"workspace": FAKE, "workspace_bytes": 1}, 0),
])
def test_i8_scaled_validation(kw, status):
    assert m.validate_i8_scaled(**i8_scaled_args(**kw)) == status


def grad_i8_args(**kw):
    a = dict(dtypeA="bf16", layoutA="k_contig", M=8, N=32, K=48, A=FAKE, lda=48, Q=FAKE, ldq=32, scaleK=FAKE, C=None,
             D=FAKE, ldd=32, dtypeD="bf16", beta=0.0, workspace=None, workspace_bytes=0)
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,status", [
    ({}, 0), ({"dtypeD": "f32"}, 0), ({"dtypeA": "f16", "dtypeD": "f16"}, 0), ({"dtypeA": "f16", "dtypeD": "f32"}, 0),
    ({"dtypeD": "f16"}, 4), ({"dtypeA": "f32", "dtypeD": "f32"}, 4), ({"dtypeA": "i8"}, 4), ({"layoutA": 5}, 4),
    ({"M": -1}, 2), ({"N": -1}, 2), ({"K": -1}, 2), ({"K": 1 << 31}, 2),
    ({"beta": float("nan"), "C": FAKE}, 10), ({"beta": 1e39, "C": FAKE}, 10),
    ({"beta": 1.0}, 1), ({"beta": 1.0, "C": FAKE}, 0),
    ({"A": None}, 1), ({"Q": None}, 1), ({"scaleK": None}, 1), ({"D": None}, 1),
    ({"M": 0, "D": None}, 0), ({"K": 0, "A": None, "Q": None, "scaleK": None, "lda": 1}, 0),
    ({"lda": 47}, 3), ({"ldq": 31}, 3), ({"ldd": 31}, 3), ({"layoutA": "mn_contig", "lda": 7}, 3),
    ({"layoutA": "mn_contig", "lda": 8}, 0),
    ({"A": FAKE + 1}, 5), ({"D": FAKE + 1}, 5), ({"C": FAKE + 1, "beta": 1.0}, 5), ({"scaleK": FAKE + 2}, 5),
    ({"Q": FAKE + 1}, 0), ({"workspace": FAKE + 4, "workspace_bytes": 64}, 5), ({"workspace_bytes": -1}, 2),
])
def test_grad_i8_validation(kw, status):
    assert m.validate_grad_i8(**grad_i8_args(**kw)) == status


@pytest.mark.parametrize("fn,args,kw,status", [
    ("rmsnorm_quant", rmsnorm_quant_args, {"X": None}, 1),
    ("rmsnorm_backward", rmsnorm_backward_args, {"workspace": None}, 11),
    ("gemm_i8_scaled", i8_scaled_args, {"K": 131072, "lda": 131072, "ldb": 131072}, 2),
    ("gemm_grad_i8", grad_i8_args, {"dtypeD": "f16"}, 4),
])
def test_entry_points_refuse_before_touching_the_device(fn, args, kw, status):
    with pytest.raises(m.MCGError) as e:
        getattr(m, fn)(**args(**kw), stream=0)
    assert e.value.status == status
    with pytest.raises(m.MCGError) as e:
        m.quantize_rows("i8", 1, 1, FAKE, 1, FAKE, 1, FAKE, stream=0)
    assert e.value.status == 4
    with pytest.raises(m.MCGError) as e:
        m.dequantize_rows("f32", 1, 8, FAKE, 7, FAKE, FAKE, 8, stream=0)
    assert e.value.status == 3


def test_workspace_queries():
    assert m.rmsnorm_backward_workspace_bytes(0, 64) == 0 and m.rmsnorm_backward_workspace_bytes(5, 0) == 0
    for M in (1, 7, 100000):
        need = m.rmsnorm_backward_workspace_bytes(M, 96)
        assert need % (96 * 4) == 0 and 0 < need <= M * 96 * 4
    # nothing to cut, empty products, and sizes that a call refuses
    assert m.i8_scaled_workspace_bytes("k_contig", 8192, 8192, 8192, FAKE, 8192, FAKE, 8192) == 0
    assert m.i8_scaled_workspace_bytes("k_contig", 0, 8, 8, FAKE, 8, FAKE, 8) == 0
    assert m.i8_scaled_workspace_bytes("k_contig", 8, 8, 200000, FAKE, 200000, FAKE, 200000) == 0
    assert m.i8_scaled_workspace_bytes("k_contig", 128, 256, 16384, FAKE, 16384, FAKE, 16384) > 0
    # Q widened once: a panel of all its columns (two for a binary32 result)
    one = 8192 * 8192 * 2
    assert m.grad_i8_workspace_bytes("bf16", "mn_contig", 8192, 8192, 8192, FAKE, 8192, FAKE, 8192, "bf16") == one
    assert m.grad_i8_workspace_bytes("bf16", "mn_contig", 8192, 8192, 8192, FAKE, 8192, FAKE, 8192, "f32") == 2 * one
    # operands without 16-byte chunks: copies of both
    assert m.i8_scaled_workspace_bytes("k_contig", 4000, 4001, 4003, FAKE, 4003, FAKE, 4003) >= (4000 + 4001) * 4016
    assert m.grad_i8_workspace_bytes("bf16", "mn_contig", 256, 256, 8192, FAKE, 256, FAKE, 256, "f32") > 0
    assert m.grad_i8_workspace_bytes("f32", "mn_contig", 256, 256, 8192, FAKE, 256, FAKE, 256, "f32") == 0


def test_operands_that_the_gpu_tests_take_in_panels():
    # (so that tests/test_gpu_linear8.py covers the copies and the widened panels)
    for M, N, K in ((600, 1300, 2050), (1300, 700, 1999), (1001, 2003, 3001)):
        for layout, ldb in (("k_contig", K + 7), ("mn_contig", N + 7)):
            assert m.i8_scaled_workspace_bytes(layout, M, N, K, FAKE, K + 5, FAKE, ldb) >= (M + N) * K
    for M, N, K in ((512, 1536, 4096), (600, 900, 700), (1001, 1103, 901)):
        for layout, lda in (("k_contig", K), ("mn_contig", M)):
            assert m.grad_i8_workspace_bytes("bf16", layout, M, N, K, FAKE, lda, FAKE, N, "bf16") >= 2 * K * N
    for layout, lda in (("k_contig", 1033), ("mn_contig", 4090)):
        assert m.grad_i8_workspace_bytes("bf16", layout, 4090, 4090, 1033, FAKE, lda, FAKE, 4090, "f32") >= 4 * 1033 * 4090


def test_arguments_that_are_none_of_the_accepted_kinds():
    kw = rmsnorm_quant_args(stream=0)
    for bad, error in (({"X": "x"}, AttributeError), ({"M": 1.5}, TypeError), ({"dtype": "f17"}, KeyError), ({"eps": "1"}, TypeError),
                       ({"M": 1 << 70}, OverflowError), ({"stream": "s"}, (TypeError, ValueError)), ({"M": "1", "X": "x"}, TypeError)):
        with pytest.raises(error):
            m.rmsnorm_quant(**{**kw, **bad})
    with pytest.raises(TypeError):
        m.quantize_rows("bf16", 1, 8, FAKE)


def test_one_copy_of_the_library_is_loaded():
    with open("/proc/self/maps") as f:
        files = {line.split()[-1] for line in f if "_libmcg.so" in line}
    assert files == {m.LIB_PATH}


def test_symbols_have_their_arguments_declared():
    lib = ctypes.CDLL(m.LIB_PATH)
    for fn in ("rmsnorm_quant", "rmsnorm_backward", "quantize_rows", "dequantize_rows", "gemm_i8_scaled",
               "gemm_grad_i8"):
        assert hasattr(lib, fn) and fn in m.EXPORTS and getattr(m.lib(), fn).argtypes
