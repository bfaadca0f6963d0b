"""Race check of the kernels for few rows, whose only meeting points are around the join of
the waves' sums in LDS, and of the second pass that takes factors apart: the library and
its build with DMP_EXTRA_SYNC (there: every wave waits for its loads and meets the others
before and after the sums are written, and after they are read) must agree bit for bit.
Groups with more rows than a pass takes use the sums' place again."""
import ctypes

import numpy as np
import pytest

from gpu_util import log
from test_gpu_ragged_race import OUT, both, handles, normal  # noqa: F401

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def offsets(counts):
    return torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int64).cuda()


# counts, K, N, B's layout, D's type: 16 and 32 columns to a workgroup; N-contiguous B
ROWS = [
    ([40, 33, 0, 80, 2, 16], 1000, 264, True, "f32"),
    ([70, 130, 5, 33] + [1] * 60, 1032, 200, True, "bf16"),
    ([1, 0, 5, 9], 4096, 512, False, "bf16"),
    ([40, 33, 0, 80, 2, 16], 1000, 264, False, "f32"),
    ([100] + [0] * 62 + [31], 520, 1032, False, "f16"),
]


@pytest.mark.parametrize("case", ROWS, ids=lambda c: f"{sum(c[0])}-{c[1]}x{c[2]}-{'col' if c[3] else 'row'}-{c[4]}")
def test_few_rows_identical_with_extra_sync(handles, case):  # noqa: F811
    counts, K, N, b_col, out = case
    log(f"[race] few rows {case}")
    T, G, off = sum(counts), len(counts), offsets(counts)
    A = normal(1, T, K).bfloat16().cuda()
    B = normal(2, G, *((N, K) if b_col else (K, N))).bfloat16().cuda()
    code, dt = OUT[out]
    for _ in range(5):
        assert both(handles, lambda: torch.zeros(T, N, dtype=dt, device="cuda"),
                    lambda lib, h, d, s: lib.gemm_run_grouped(
                        h, A.data_ptr(), B.data_ptr(), None, d.data_ptr(), off.data_ptr(), G, T, N, K, K,
                        K if b_col else N, N, 1, 2 if b_col else 0, 1.0, 0.0, code, code, s))


@pytest.mark.parametrize("low", [0, -76], ids=["ordinary", "apart"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("counts,K,N", [([40, 33, 0, 20, 2], 1000, 264), ([40, 1, 0, 33] + [1] * 60, 1000, 200),
                                        ([40, 1, 0, 33] + [1] * 60, 1000, 520), ([70, 130, 5, 300], 1000, 520),
                                        ([1700, 0, 1501, 1200], 1088, 4096)])
def test_8_bit_identical_with_extra_sync(handles, counts, K, N, out, low):  # noqa: F811
    """low: powers of two in both operands' scales (2^-76 each: taken apart)."""
    import dense_mixed_precision_02_amd as dmp
    from dense_mixed_precision_02_amd import binding
    log(f"[race] scaled8 {counts[:4]} {K}x{N} {out} {low}")
    T, G, off = sum(counts), len(counts), offsets(counts)
    a, b = dmp.quant8(normal(5, T, K).cuda()), dmp.quant8(normal(6, G, N, K).cuda(), block=128)
    a.scale *= 2.0 ** low
    b.scale *= 2.0 ** low
    kp, kb, nb = -(-K // 16) * 16, -(-K // 128), -(-N // 128)
    qa = binding.Q8Operand(a.q.data_ptr(), a.scale.data_ptr(), kp, 1, T, 0, 0, 0)
    qb = binding.Q8Operand(b.q.data_ptr(), b.scale.data_ptr(), kp, 1, nb, N * kp, kb * nb, 0)
    code, dt = OUT[out]
    for _ in range(5):
        assert both(handles, lambda: torch.zeros(T, N, dtype=dt, device="cuda"),
                    lambda lib, h, d, s: lib.gemm_run_scaled8(
                        h, ctypes.byref(qa), ctypes.byref(qb), None, d.data_ptr(), off.data_ptr(), G, T, N, K, N, 0,
                        2.0 ** 100 if low else 1.0, 0.0, code, code, s))
