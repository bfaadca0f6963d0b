"""Race check of the 256x256 tiles of the grouped products, with N-contiguous B and with whole
and cut rounds of tiles: the library and its build with DMP_EXTRA_SYNC must agree bit for
bit.  (tests/native/ragged_rules_check.cpp holds that these shapes take those tiles.)"""
import numpy as np
import pytest

from gpu_util import log
from test_gpu_ragged_race import OUT, both, handles, normal  # noqa: F401

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("b_col", [True, False], ids=["col", "row"])
@pytest.mark.parametrize("counts,K,N,out", [([1700, 0, 1501, 1200], 1088, 2048, "f32"), ([2048, 2100], 512, 4096, "bf16"),
                                            ([4400, 3, 40], 200, 4000, "f16")])
def test_large_tiles_identical_with_extra_sync(handles, counts, K, N, out, b_col):  # noqa: F811
    log(f"[race] large tiles {counts} {K}x{N} {out} {'col' if b_col else 'row'}")
    T, G = sum(counts), len(counts)
    A = normal(1, T, K).bfloat16().cuda()
    B = normal(2, G, *((N, K) if b_col else (K, N))).bfloat16().cuda()
    off = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int64).cuda()
    code, dt = OUT[out]
    for _ in range(3):
        assert both(handles, lambda: torch.zeros(T, N, dtype=dt, device="cuda"),
                    lambda lib, h, d, s: lib.gemm_run_grouped(
                        h, A.data_ptr(), B.data_ptr(), None, d.data_ptr(), off.data_ptr(), G, T, N, K, K,
                        K if b_col else N, N, 1, 2 if b_col else 0, 1.0, 0.0, code, code, s))
