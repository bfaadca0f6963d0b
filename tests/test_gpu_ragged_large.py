"""Grouped and 8-bit products whose operands pass 2^32 bytes: groups that begin there
are read and written in the right place.  Values are small integers, so results are exact
and compared for equality; the 64-bit comparison takes the first and last groups."""
import pytest

from test_gpu_grouped import dmp, offsets_of  # noqa: F401

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def ints(seed, *shape, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-2, 3, shape, generator=g, device="cuda", dtype=torch.int8).to(dtype)


@pytest.mark.parametrize("rows", [3, 200], ids=["few", "tiles"])
@pytest.mark.parametrize("b_col", [True, False], ids=["col", "row"])
def test_weights_beyond_4_gib(dmp, b_col, rows):  # noqa: F811
    G, K, N = 34, 4096, 16384  # 4.25 GiB of weights
    counts = [rows] + [0] * (G - 2) + [rows]
    A, off = ints(1, 2 * rows, K), offsets_of(counts).cuda()
    B = ints(2, G, *((N, K) if b_col else (K, N)))
    B = B.transpose(1, 2) if b_col else B
    D = dmp.gemm_grouped(A, B, off)
    for g, part in ((0, slice(0, rows)), (G - 1, slice(rows, 2 * rows))):
        assert torch.equal(D[part].double(), A[part].double() @ B[g].double())


def test_gradients_beyond_4_gib(dmp):  # noqa: F811
    G, M, N = 18, 8192, 8192  # 4.5 GiB of fp32 gradients
    counts = [70] + [0] * (G - 2) + [130]
    X, Y, off = ints(3, 200, M), ints(4, 200, N), offsets_of(counts).cuda()
    D = dmp.gemm_grouped_wgrad(X, Y, off)
    assert torch.equal(D[0], X[:70].float().t().contiguous() @ Y[:70].float())
    assert torch.equal(D[G - 1], X[70:].float().t().contiguous() @ Y[70:].float())
    assert not D[1:G - 1].any()


@pytest.mark.parametrize("rows", [3, 200], ids=["few", "tiles"])
def test_8_bit_weights_beyond_4_gib(dmp, rows):  # noqa: F811
    G, K, N = 66, 4096, 16384  # 4.1 GiB of 8-bit weights
    f8 = torch.float8_e4m3fn
    counts = [rows] + [0] * (G - 2) + [rows]
    off = offsets_of(counts).cuda()
    a, b = ints(5, 2 * rows, K, dtype=f8), ints(6, G, N, K, dtype=f8)
    sa = torch.full((2 * rows, K // 128), 0.5, device="cuda")
    sb = torch.ones(G, N // 128, K // 128, device="cuda")
    sb[G - 1] = 2.0
    D = dmp.gemm_scaled8(dmp.Scaled8(a, sa), dmp.Scaled8(b, sb, block=128), off)
    for g, part, f in ((0, slice(0, rows), 0.5), (G - 1, slice(rows, 2 * rows), 1.0)):
        assert torch.equal(D[part].double(), f * (a[part].double() @ b[g].double().t().contiguous()))


def test_quantization_beyond_4_gib(dmp):  # noqa: F811
    """The last rows of a 4.25 GiB matrix: as quantized alone."""
    X = torch.zeros(557056, 4096, dtype=torch.bfloat16, device="cuda")
    tail = ints(7, 300, 4096)
    X[-300:] = tail
    for block, rows in ((1, 300), (128, 256)):
        whole, part = dmp.quant8(X, block=block), dmp.quant8(tail[300 - rows:], block=block)
        assert torch.equal(whole.q[-rows:].view(torch.uint8), part.q.view(torch.uint8))
        assert torch.equal(whole.scale[-(-(-rows // block)):], part.scale)
