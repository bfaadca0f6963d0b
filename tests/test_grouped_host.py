"""Host-side checks of the grouped and 8-bit entry points: refusals of the C ABI
(a NULL handle makes no HIP call; the argument checks themselves run under the
sanitizers in a small C++ program) and of the torch front ends, on the CPU."""
import ctypes
import os

import pytest

import dense_mixed_precision_02_amd as dmp
from test_sanitizers import NATIVE, build_and_run

torch = pytest.importorskip("torch")


def test_argument_checks_under_sanitizers(tmp_path):
    out = build_and_run(tmp_path, "g++", [os.path.join(NATIVE, "ragged_plan_check.cpp")], ["-std=c++17"],
                        "ragged_plan_check")
    assert "0 failures" in out


def test_null_handle_is_refused():
    lib = dmp.load_library()
    assert lib.gemm_run_grouped(None, 0, 0, 0, 0, 0, 1, 1, 1, 1, 1, 1, 1, 0, 0, 1.0, 0.0, 0, 0, 0) == 1
    assert lib.gemm_run_grouped_wgrad(None, 0, 0, 0, 0, 0, 1, 1, 1, 1, 1, 1, 1, 0, 0, 1.0, 0.0, 0, 0, 0) == 1
    assert lib.gemm_quant8(None, 0, 1, 1, 1, 0, 0, 1, 1, 0, 0, 0, 0) == 1
    o = dmp.Q8Operand()
    assert lib.gemm_run_scaled8(None, ctypes.byref(o), ctypes.byref(o), 0, 0, 0, 1, 1, 1, 1, 1, 0, 1.0, 0.0,
                                0, 0, 0) == 1


def test_operand_structure_matches_the_header():
    text = open(os.path.join(os.path.dirname(NATIVE), "..", "include", "dmp_gemm.h")).read()
    body = text[text.index("typedef struct {\n    const void *q;"):text.index("} gemm_q8_t;")]
    names = [n.strip(" ;*\n") for line in body.splitlines()[1:] for n in line.split("/*")[0].replace(
        "const void", "").replace("const float", "").replace("int64_t", "").replace("int ", "").split(",")]
    assert [n for n in names if n] == [f[0] for f in dmp.Q8Operand._fields_]
    assert ctypes.sizeof(dmp.Q8Operand) == 64


def test_front_ends_refuse_what_they_do_not_take():
    f16, f32, i8 = (lambda *s: torch.zeros(*s, dtype=torch.float16)), (lambda *s: torch.zeros(*s)), \
        (lambda *s: torch.zeros(*s, dtype=torch.int8))
    off = torch.zeros(3, dtype=torch.int64)
    for A, B in ((f32(4, 8), f32(2, 8, 8)), (f16(4, 8), f32(2, 8, 8)), (i8(4, 8), i8(2, 8, 8))):
        with pytest.raises(TypeError):
            dmp.gemm_grouped(A, B, off)
        with pytest.raises(TypeError):
            dmp.gemm_grouped_wgrad(A, B, off)
    with pytest.raises(ValueError):  # not on a GPU
        dmp.gemm_grouped(f16(4, 8), f16(2, 8, 8), off)
    with pytest.raises(ValueError):
        dmp.gemm_grouped_wgrad(f16(4, 8), f16(4, 8), off)
    with pytest.raises(ValueError):
        dmp.quant8(f16(4, 8))
    with pytest.raises(TypeError):
        dmp.quant8(i8(4, 8))
    with pytest.raises(TypeError):
        dmp.quant8(f16(4, 8), dtype=torch.float16)
    q, s = torch.zeros(4, 16).to(torch.float8_e4m3fn), f32(4, 1)
    with pytest.raises(ValueError):  # not on a GPU
        dmp.Scaled8(q, s)
    with pytest.raises(TypeError):
        dmp.Scaled8(f16(4, 16), s)
    with pytest.raises(ValueError):
        dmp.Scaled8(q, s, block=64)
    with pytest.raises(ValueError):  # K = 17 needs rows of 32
        dmp.Scaled8(q, s, K=17)
    with pytest.raises(ValueError):
        dmp.Scaled8(q, f32(4, 2))
