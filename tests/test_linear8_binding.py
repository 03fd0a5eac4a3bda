"""The binding of the 8-bit linear layer without its C extension (not built, or built
for another Python): the same calls, refusals and conversions through ctypes."""
import importlib.util
import os
import subprocess
import sys

import pytest

m = pytest.importorskip("matrix_core_gemm_amd")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # aligned and non-null; never dereferenced here


def call_both(name, *args):
    """Status or error type of a refused call through the C extension and through ctypes."""
    out = []
    for side in (m._mcgcall, m._CtypesCalls()):
        try:
            out.append(getattr(side, name)(*args))
        except Exception as e:
            out.append(type(e))
    return out


class Tensor:
    nbytes = 12345

    def data_ptr(self):
        return FAKE


QUANT = ["bf16", 4, 64, FAKE, 64, None, 0, None, 1e-5, None, 0, FAKE, 64, FAKE, None, 0]
BACK = ["bf16", "bf16", 4, 64, FAKE, 64, FAKE, 64, None, None, FAKE, None, 0, FAKE, 64, FAKE, None, 0, 0]
ROWS = ["bf16", 4, 64, FAKE, 64, FAKE, 64, FAKE, 0]
BACKROWS = ["bf16", 4, 64, FAKE, 64, FAKE, FAKE, 64, 0]
SCALED = ["k_contig", 8, 32, 48, FAKE, 48, FAKE, FAKE, 48, FAKE, None, FAKE, 32, "bf16", None, 0, 0]
GRAD = ["bf16", "k_contig", 8, 32, 48, FAKE, 48, FAKE, 32, FAKE, None, FAKE, 32, "bf16", 0.0, None, 0, 0]


# every call is refused: no argument reaches a device
@pytest.mark.parametrize("name,args,changes,expect", [
    ("rmsnorm_quant", QUANT, {3: None}, 1), ("rmsnorm_quant", QUANT, {1: -1}, 2), ("rmsnorm_quant", QUANT, {4: 63}, 3),
    ("rmsnorm_quant", QUANT, {0: "i8"}, 4), ("rmsnorm_quant", QUANT, {0: 42}, 4), ("rmsnorm_quant", QUANT, {13: FAKE + 2}, 5),
    ("rmsnorm_quant", QUANT, {8: -1.0}, 10), ("rmsnorm_quant", QUANT, {8: "1"}, TypeError), ("rmsnorm_quant", QUANT, {0: "f17"}, KeyError),
    ("rmsnorm_quant", QUANT, {1: 1.5}, TypeError), ("rmsnorm_quant", QUANT, {1: 1 << 70}, OverflowError),
    ("rmsnorm_quant", QUANT, {3: "x"}, AttributeError), ("rmsnorm_quant", QUANT, {3: Tensor(), 13: None}, 1),
    ("rmsnorm_backward", BACK, {}, 11), ("rmsnorm_backward", BACK, {16: FAKE, 17: 4 * 64 * 4 - 1}, 11),
    ("rmsnorm_backward", BACK, {1: "i8"}, 1), ("rmsnorm_backward", BACK, {16: FAKE, 17: -1}, 2), ("rmsnorm_backward", BACK, {1: "f16"}, 4),
    ("rmsnorm_backward", BACK, {16: Tensor(), 14: 63}, 3), ("rmsnorm_backward", BACK, {10: FAKE + 1, 16: Tensor()}, 5),
    ("quantize_rows", ROWS, {7: None}, 1), ("quantize_rows", ROWS, {6: 63}, 3), ("quantize_rows", ROWS[:-1], {}, TypeError),
    ("dequantize_rows", BACKROWS, {6: None}, 1), ("dequantize_rows", BACKROWS, {7: 63}, 3), ("dequantize_rows", BACKROWS, {0: "i32"}, 4),
    ("gemm_i8_scaled", SCALED, {3: 131072, 5: 131072, 8: 131072}, 2), ("gemm_i8_scaled", SCALED, {0: "mn_contig", 8: 31}, 3),
    ("gemm_i8_scaled", SCALED, {13: "i8"}, 4), ("gemm_i8_scaled", SCALED, {14: FAKE + 4, 15: 64}, 5), ("gemm_i8_scaled", SCALED, {0: "row"}, KeyError),
    ("gemm_grad_i8", GRAD, {9: None}, 1), ("gemm_grad_i8", GRAD, {13: "f16"}, 4), ("gemm_grad_i8", GRAD, {14: 1.0}, 1),
    ("gemm_grad_i8", GRAD, {14: float("nan")}, 10), ("gemm_grad_i8", GRAD, {12: 31}, 3), ("gemm_grad_i8", GRAD, {16: -1, 15: FAKE}, 2),
])
def test_the_same_refusals_with_and_without_the_extension(name, args, changes, expect):
    args = list(args)
    for i, v in changes.items():
        args[i] = v
    assert call_both(name, *args) == [expect, expect]


def test_the_package_works_without_the_extension():
    code = """
import sys
sys.modules["matrix_core_gemm_amd._mcgcall"] = None   # what importing an absent module does
import matrix_core_gemm_amd as m
assert isinstance(m._mcgcall, m._CtypesCalls)
F = 0x10000
for fn, status in ((lambda: m.rmsnorm_quant("bf16", 4, 64, None, 64, None, 0, None, 1e-5, None, 0, F, 64, F, stream=0), 1),
                   (lambda: m.rmsnorm_backward("bf16", "bf16", 4, 64, F, 64, F, 64, None, None, F, None, 0, F, 64, F, stream=0), 11),
                   (lambda: m.quantize_rows("i8", 1, 1, F, 1, F, 1, F, stream=0), 4),
                   (lambda: m.dequantize_rows("f32", 1, 8, F, 7, F, F, 8, stream=0), 3),
                   (lambda: m.gemm_i8_scaled("k_contig", 8, 32, 200000, F, 200000, F, F, 200000, F, None, F, 32, "bf16", stream=0), 2),
                   (lambda: m.gemm_grad_i8("bf16", "k_contig", 8, 32, 48, F, 48, F, 32, F, None, F, 32, "bf16", float("inf"), stream=0), 10)):
    try:
        fn()
    except m.MCGError as e:
        assert e.status == status, (e, status)
    else:
        raise AssertionError(status)
# an empty product is no call of the device: it succeeds
m.gemm_i8_scaled("k_contig", 0, 32, 48, None, 48, None, None, 48, None, None, None, 32, "bf16", stream=0)
print("ok")
"""
    p = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0 and p.stdout.strip().endswith("ok"), p.stderr


def load_build():
    spec = importlib.util.spec_from_file_location("_build_under_test", os.path.join(ROOT, "matrix_core_gemm_amd", "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    return b


def test_a_build_without_a_c_compiler_says_so_and_leaves_no_old_extension(tmp_path, monkeypatch, capsys):
    b = load_build()
    monkeypatch.setattr(b, "HERE", str(tmp_path))
    monkeypatch.setattr(b, "CALL", str(tmp_path / os.path.basename(b.CALL)))
    monkeypatch.setattr(b, "CC", "no-such-compiler")
    for name in (os.path.basename(b.CALL), "_mcgcall.so"):
        (tmp_path / name).write_text("an older build")
    assert b.build_call() is None
    assert "ctypes" in capsys.readouterr().err and os.listdir(tmp_path) == []


def test_the_extension_is_named_for_its_python():
    import sysconfig
    assert os.path.basename(load_build().CALL) == "_mcgcall" + sysconfig.get_config_var("EXT_SUFFIX")
