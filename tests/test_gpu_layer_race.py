"""Race check of the adapters and the 8-bit gradients: the library and its build with
DMP_EXTRA_SYNC (every pipeline step waits for its loads and meets every wave, the
arithmetic unchanged) must give bit-identical results on the same inputs, for every
kernel."""
import ctypes
import os

import pytest

from gpu_util import log

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

PKG = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dense_mixed_precision_02_amd")
LIBS = [os.path.join(PKG, "libdmp_gemm.so"), os.path.join(PKG, "libdmp_gemm_sync.so")]
OUT = {"f32": (0, torch.float32), "f16": (1, torch.float16), "bf16": (2, torch.bfloat16)}


@pytest.fixture(scope="module")
def handles():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from dense_mixed_precision_02_amd import binding
    main = binding.load_library()
    out = []
    for path in LIBS:
        lib = ctypes.CDLL(path)
        for name in ("gemm_create", "gemm_destroy", "gemm_adapters_work", "gemm_run_adapters", "gemm_wgrad8_work", "gemm_run_wgrad8"):
            getattr(lib, name).argtypes = getattr(main, name).argtypes
            getattr(lib, name).restype = getattr(main, name).restype
        h = ctypes.c_void_p()
        assert lib.gemm_create(ctypes.byref(h)) == 0
        out.append((lib, h))
    yield out
    for lib, h in out:
        lib.gemm_destroy(h)


def normal(seed, *shape, dtype):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype).cuda()


def bits(x):
    return x.view(torch.int32 if x.element_size() == 4 else torch.int16)


# rows, requests, K, N, rank, linear, D's type, an element's shift of X (no 16-byte granules)
ADAPTERS = [
    (8200, 5, 200, 2048, 72, True, "bf16", 0),    # 256 x 256 tiles
    (8200, 5, 264, 2048, 16, False, "f32", 0),
    (1100, 40, 264, 4104, 24, True, "f32", 0),    # 128 x 128
    (1100, 40, 264, 4104, 24, False, "bf16", 0),
    (900, 40, 1000, 520, 24, True, "f32", 0),     # 64 x 64
    (900, 40, 1000, 520, 24, False, "bf16", 0),
    (900, 40, 1000, 520, 13, True, "f16", 0),
    (900, 40, 1003, 517, 13, False, "f32", 1),    # any alignment
    (900, 40, 1003, 517, 13, True, "bf16", 1),
    (64, 64, 4096, 1024, 16, True, "bf16", 0),    # few rows
    (120, 30, 1000, 264, 40, True, "f32", 0),
    (120, 30, 1003, 517, 13, False, "f32", 1),
    (5, 5, 512, 520, 8, True, "f16", 0),
]


@pytest.mark.parametrize("case", ADAPTERS, ids=lambda c: f"{c[0]}x{c[2]}x{c[3]}r{c[4]}-{'linear' if c[5] else 'row'}-{c[6]}")
def test_adapters(handles, case):
    from dense_mixed_precision_02_amd import binding
    T, S, K, N, r, linear, out, shift = case
    log(f"[race adapters] {case}")
    a = 4
    dt = torch.bfloat16 if out != "f16" else torch.float16
    X = normal(1, T * K + 8, dtype=dt)
    W, A, B = normal(2, N * K, dtype=dt), normal(3, a * r * K, dtype=dt), normal(4, a * N * r, dtype=dt)
    off = torch.tensor([T * i // S for i in range(S + 1)], device="cuda")
    ids = torch.tensor([i % (a + 1) - 1 for i in range(S)], dtype=torch.int32, device="cuda")
    ops = binding.AdapterOperands(A.data_ptr(), B.data_ptr(), ids.data_ptr(), None, a, r, K if linear else r, r if linear else N)
    flags = binding.GEMM_B_COLMAJOR | binding.GEMM_ADAPTER_A_COLMAJOR if linear else 0
    res = []
    for lib, h in handles:
        D = torch.zeros(T, N, dtype=OUT[out][1], device="cuda")
        hidden = torch.zeros(T, r, dtype=dt, device="cuda")
        work = torch.empty(lib.gemm_adapters_work(h, X.data_ptr() + 2 * shift, W.data_ptr(), S, T, N, K, r, K, K if linear else N,
                                                  OUT[out][0], flags), dtype=torch.uint8, device="cuda")
        rc = lib.gemm_run_adapters(h, X.data_ptr() + 2 * shift, W.data_ptr(), ctypes.byref(ops), None, D.data_ptr(),
                                   off.data_ptr(), S, T, N, K, K, K if linear else N, N, 0 if dt == torch.float16 else 1, flags, 1.0,
                                   0.0, 0, OUT[out][0], hidden.data_ptr(), r, work.data_ptr(),
                                   torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        torch.cuda.synchronize()
        res.append((bits(D), bits(hidden)))
    assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])


# rows, groups (0: one of all rows), M, N, Y's type, D's type, an element's shift of Y
WGRAD = [
    (1000, 0, 4096, 4096, "bf16", "bf16", 0),   # 256 x 256 tiles
    (2100, 5, 2048, 2056, "f16", "f32", 0),
    (3000, 7, 520, 264, "bf16", "f32", 0),      # 64 x 128
    (9000, 0, 200, 136, "f16", "f16", 0),       # split rows
    (5000, 4, 1000, 520, "bf16", "f32", 0),     # 128 x 128
    (9000, 0, 2048, 2048, "f16", "bf16", 0),    # 256 x 256, split rows
    (3000, 7, 131, 99, "bf16", "bf16", 1),      # any alignment
]


@pytest.mark.parametrize("case", WGRAD, ids=lambda c: f"{c[0]}g{c[1]}-{c[2]}x{c[3]}-{c[5]}")
def test_wgrad8(handles, case):
    import dense_mixed_precision_02_amd as dmp
    T, G, M, N, yt, out, shift = case
    log(f"[race wgrad8] {case}")
    dt = OUT[yt][1]
    x = dmp.quant8(normal(1, T, M, dtype=dt), pow2=True)
    Y = normal(2, T * N + 8, dtype=dt)
    g = max(G, 1)
    off = torch.tensor([T * i // g for i in range(g + 1)], device="cuda")
    res = []
    for lib, h in handles:
        D = torch.zeros(g, M, N, dtype=OUT[out][1], device="cuda")
        need = lib.gemm_wgrad8_work(h, Y.data_ptr() + 2 * shift, g, M, N, T, N)
        work = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
        rc = lib.gemm_run_wgrad8(h, ctypes.byref(x.operand), Y.data_ptr() + 2 * shift, None, D.data_ptr(),
                                 off.data_ptr() if G else None, g, M, N, T, N, N, 0 if yt == "f16" else 1, 0, 1.0, 0.0, 0,
                                 OUT[out][0], work.data_ptr(), torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        torch.cuda.synchronize()
        res.append(bits(D))
    assert torch.equal(*res)
