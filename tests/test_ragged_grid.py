"""Grids of the grouped and 8-bit kernels, on the CPU (see tests/native/ragged_grid_check.cpp)."""
import os

from test_sanitizers import NATIVE, build_and_run


def test_grid_shapes_under_sanitizers(tmp_path):
    out = build_and_run(tmp_path, "g++", [os.path.join(NATIVE, "ragged_grid_check.cpp")], ["-std=c++17"],
                        "ragged_grid_check")
    assert "0 failures" in out
