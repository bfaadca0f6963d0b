"""Race check of the products over ragged groups and of the 8-bit products: the
library and its build with DMP_EXTRA_SYNC (every pipeline step waits for its loads
and meets every wave, the arithmetic unchanged) must give bit-identical results on
the same inputs, for every kernel and layout: 256x256 tiles (whole and cut), staged
tiles, the staged kernel for any alignment, few rows, and both 8-bit tiles."""
import ctypes
import os

import numpy as np
import pytest

from gpu_util import log

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(HERE, "dense_mixed_precision_02_amd")
LIBS = [os.path.join(PKG, "libdmp_gemm.so"), os.path.join(PKG, "libdmp_gemm_sync.so")]
OUT = {"f32": (0, torch.float32), "f16": (1, torch.float16), "bf16": (2, torch.bfloat16)}


@pytest.fixture(scope="module")
def handles():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from dense_mixed_precision_02_amd import binding
    i64, vp, ci, cu, cf = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_uint, ctypes.c_float
    q8 = ctypes.POINTER(binding.Q8Operand)
    out = []
    for path in LIBS:
        lib = ctypes.CDLL(path)
        lib.gemm_create.argtypes = [ctypes.POINTER(vp)]
        lib.gemm_destroy.argtypes = [vp]
        for f in (lib.gemm_run_grouped, lib.gemm_run_grouped_wgrad):
            f.argtypes = [vp] * 6 + [i64] * 7 + [ci, cu, cf, cf, ci, ci, vp]
        lib.gemm_run_scaled8.argtypes = [vp, q8, q8, vp, vp, vp] + [i64] * 5 + [cu, cf, cf, ci, ci, vp]
        h = vp()
        assert lib.gemm_create(ctypes.byref(h)) == 0
        out.append((lib, h))
    yield out
    for lib, h in out:
        lib.gemm_destroy(h)


def normal(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g)


def both(handles, make, call):
    """Bit patterns of the results of the two libraries."""
    res = []
    for lib, h in handles:
        d = make()
        assert call(lib, h, d, torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        res.append(d.view(torch.int32 if d.element_size() == 4 else torch.int16))
    return torch.equal(*res)


# counts, K, N, B's layout, D's type, an element's shift of A (no 16-byte granules)
ROWS = [
    ([1700, 0, 1501, 1200], 1088, 1024, True, "bf16", 0),
    ([1700, 0, 1501, 1200], 1088, 1024, False, "f32", 0),
    ([2048, 2100], 512, 4096, True, "f32", 0),
    ([70, 130, 5, 300], 1000, 520, True, "f16", 0),
    ([70, 130, 5, 300], 1000, 520, False, "bf16", 0),
    ([70, 130, 5, 300], 1003, 517, False, "f32", 1),
    ([70, 130, 5, 300], 1003, 517, True, "f32", 1),
    ([1, 0, 5, 9], 4096, 512, True, "bf16", 0),
    ([40, 33, 80, 2], 4096, 512, True, "bf16", 0),
]


@pytest.mark.parametrize("case", ROWS, ids=lambda c: f"{sum(c[0])}-{c[1]}x{c[2]}-{'col' if c[3] else 'row'}-{c[4]}")
def test_grouped_identical_with_extra_sync(handles, case):
    counts, K, N, b_col, out, shift = case
    log(f"[race] grouped {case}")
    T, G = sum(counts), len(counts)
    A = normal(1, T * K + 8).bfloat16().cuda()[shift:]
    B = normal(2, G, *((N, K) if b_col else (K, N))).bfloat16().cuda()
    off = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int64).cuda()
    code, dt = OUT[out]
    assert both(handles, lambda: torch.zeros(T, N, dtype=dt, device="cuda"),
                lambda lib, h, d, s: lib.gemm_run_grouped(
                    h, A.data_ptr(), B.data_ptr(), None, d.data_ptr(), off.data_ptr(), G, T, N, K, K,
                    K if b_col else N, N, 1, 2 if b_col else 0, 1.0, 0.0, code, code, s))


@pytest.mark.parametrize("counts,M,N", [([1700, 3, 1501, 1200], 2048, 2048), ([300, 0, 129, 64], 520, 1032),
                                        ([300, 0, 129, 65], 517, 1031)])
def test_wgrad_identical_with_extra_sync(handles, counts, M, N):
    log(f"[race] wgrad {counts} {M}x{N}")
    T, G = sum(counts), len(counts)
    X, Y = normal(3, T, M).bfloat16().cuda(), normal(4, T, N).bfloat16().cuda()
    off = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int64).cuda()
    assert both(handles, lambda: torch.zeros(G, M, N, device="cuda"),
                lambda lib, h, d, s: lib.gemm_run_grouped_wgrad(
                    h, X.data_ptr(), Y.data_ptr(), None, d.data_ptr(), off.data_ptr(), G, M, N, T, M, N, N,
                    1, 0, 1.0, 0.0, 0, 0, s))


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("counts,K,N", [([1700, 0, 1501, 1200], 1088, 4096), ([70, 130, 5, 300], 1000, 520),
                                        ([1, 0, 5, 9], 4096, 512)])
def test_scaled8_identical_with_extra_sync(handles, counts, K, N, out):
    import dense_mixed_precision_02_amd as dmp
    from dense_mixed_precision_02_amd import binding
    log(f"[race] scaled8 {counts} {K}x{N} {out}")
    T, G = sum(counts), len(counts)
    a = dmp.quant8(normal(5, T, K).cuda(), block=1)
    b = dmp.quant8(normal(6, G, N, K).cuda(), block=128)
    off = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int64).cuda()
    kp, kb, nb = -(-K // 16) * 16, -(-K // 128), -(-N // 128)
    qa = binding.Q8Operand(a.q.data_ptr(), a.scale.data_ptr(), kp, 1, T, 0, 0, 0)
    qb = binding.Q8Operand(b.q.data_ptr(), b.scale.data_ptr(), kp, 1, nb, N * kp, kb * nb, 0)
    code, dt = OUT[out]
    assert both(handles, lambda: torch.zeros(T, N, dtype=dt, device="cuda"),
                lambda lib, h, d, s: lib.gemm_run_scaled8(
                    h, ctypes.byref(qa), ctypes.byref(qb), None, d.data_ptr(), off.data_ptr(), G, T, N, K, N, 0,
                    1.0, 0.0, code, code, s))
