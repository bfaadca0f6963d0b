"""Which kernel the grouped and 8-bit calls take, on the CPU (see
tests/native/ragged_rules_check.cpp)."""
import os

from test_sanitizers import NATIVE, build_and_run


def test_kernel_rules_under_sanitizers(tmp_path):
    out = build_and_run(tmp_path, "g++", [os.path.join(NATIVE, "ragged_rules_check.cpp")], ["-std=c++17"],
                        "ragged_rules_check")
    assert "0 failures" in out
