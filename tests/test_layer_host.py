"""Host-side checks of the adapters, the 8-bit gradients and the router: argument
checks and kernel choice under the sanitizers in a small C++ program, refusals of the
C ABI without a handle and of the torch front ends, on the CPU."""
import ctypes
import os

import pytest

import dense_mixed_precision_02_amd as dmp
from test_sanitizers import NATIVE, build_and_run

torch = pytest.importorskip("torch")


def test_argument_checks_and_rules_under_sanitizers(tmp_path):
    out = build_and_run(tmp_path, "g++", [os.path.join(NATIVE, "layer_plan_check.cpp")], ["-std=c++17"],
                        "layer_plan_check")
    assert "0 failures" in out


def test_null_handle_is_refused():
    lib = dmp.load_library()
    a, q = dmp.AdapterOperands(), dmp.Q8Operand()
    assert lib.gemm_adapters_work(None, 0, 0, 1, 1, 1, 1, 1, 1, 1, 0, 0) == -1
    assert lib.gemm_run_adapters(None, 0, 0, ctypes.byref(a), 0, 0, 0, 1, 1, 1, 1, 1, 1, 1, 0, 0, 1.0, 0.0, 0, 0, 0, 0, 0,
                                 0) == 1
    assert lib.gemm_wgrad8_work(None, 0, 1, 1, 1, 1, 1) == -1
    assert lib.gemm_run_wgrad8(None, ctypes.byref(q), 0, 0, 0, 0, 1, 1, 1, 1, 1, 1, 0, 0, 1.0, 0.0, 0, 0, 0, 0) == 1


def test_structures_match_the_header():
    text = open(os.path.join(os.path.dirname(NATIVE), "..", "include", "dmp_gemm.h")).read()
    for name, struct, size in (("gemm_adapters_t", dmp.AdapterOperands, 64), ("gemm_route_t", dmp.RouteTables, 64)):
        end = text.index("} " + name + ";")
        body = text[text.rindex("typedef struct {", 0, end):end]
        names = [n.split("/*")[0].strip(" ;*\n").split()[-1].strip("*") for line in body.splitlines()[1:] if line.strip()
                 for n in line.split("/*")[0].split(",") if n.strip(" ;")]
        assert names == [f[0] for f in struct._fields_], name
        assert ctypes.sizeof(struct) == size


def test_front_ends_refuse_what_they_do_not_take():
    h = torch.float16
    X, W, A, B = torch.zeros(4, 8, dtype=h), torch.zeros(8, 8, dtype=h), torch.zeros(2, 8, 4, dtype=h), torch.zeros(2, 4, 8, dtype=h)
    off = torch.tensor([0, 2, 4])
    with pytest.raises(ValueError, match="GPU"):
        dmp.gemm_adapters(X, W, A, B, off)
    with pytest.raises(TypeError):
        dmp.gemm_adapters(X.float(), W.float(), A, B, off)
    with pytest.raises(TypeError):
        dmp.gemm_adapters(X, W.bfloat16(), A, B, off)
    q, s = torch.zeros(4, 16, dtype=torch.uint8).view(torch.float8_e4m3fn), torch.zeros(4, 1)
    with pytest.raises(ValueError):  # not on a GPU
        dmp.gemm_wgrad8(dmp.Scaled8(q, s), X)
