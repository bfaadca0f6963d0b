"""Grouped and 8-bit calls of 2^24 workgroups and more, which as one row of 256 threads
each would pass the 2^32 - 1 threads that a launch takes along an axis.  Values are small
integers, so every result is exact."""
import pytest

from test_gpu_grouped import dmp, offsets_of  # noqa: F401

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def ints(seed, *shape, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-2, 3, shape, generator=g, device="cuda", dtype=torch.int8).to(dtype)


@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("extra", [0, 5], ids=["full", "ragged"])
def test_quantization_of_many_batch_entries(dmp, block, extra):  # noqa: F811
    n = (1 << 24) + extra
    X = ints(1, n, 1, 16)
    r = dmp.quant8(X, block=block)
    a = X.view(n, 16).float().abs().amax(1).clamp_min(2.0 ** -100)
    assert torch.equal(r.scale.view(n), a / torch.tensor(448.0, device="cuda"))
    # |x| is the largest magnitude, half of it or zero: the 8-bit values are 448, 224 and 0
    assert torch.equal(r.q.view(n, 16).float(), X.view(n, 16).float() * 448.0 / a[:, None])


@pytest.mark.parametrize("b_col,N", [(True, 544), (False, 2056)], ids=["col", "row"])
def test_products_of_many_groups(dmp, b_col, N):  # noqa: F811
    """2^20 groups of 17 column blocks each, one of a thousand groups with rows."""
    G, K = 1 << 20, 8
    rows = torch.zeros(G, dtype=torch.int64)
    rows[::1000], rows[-1] = 1, 2
    used = rows.nonzero().view(-1)
    off, T = offsets_of(rows.tolist()).cuda(), int(rows.sum())
    A = ints(2, T, K)
    B = ints(3, *((G, N, K) if b_col else (G, K, N)))
    B = B.transpose(1, 2) if b_col else B
    out = torch.full((T, N), 7.0, device="cuda")
    dmp.gemm_grouped(A, B, off, out=out)
    group = torch.repeat_interleave(used, rows[used]).cuda()
    want = torch.bmm(A.float()[:, None], B[group].float().contiguous())[:, 0]
    assert torch.equal(out, want)


def test_8_bit_products_of_many_groups(dmp):  # noqa: F811
    G, K, N = 1 << 20, 16, 1032  # 17 blocks of 64 columns
    rows = torch.zeros(G, dtype=torch.int64)
    rows[::1000], rows[-1] = 1, 2
    used = rows.nonzero().view(-1)
    off, T = offsets_of(rows.tolist()).cuda(), int(rows.sum())
    f8 = torch.float8_e4m3fn
    a, b = ints(4, T, K, dtype=f8), ints(5, G, N, K, dtype=f8)
    sa, sb = torch.full((T, 1), 0.5, device="cuda"), torch.full((G, 9, 1), 2.0, device="cuda")
    out = torch.full((T, N), 7.0, device="cuda")
    dmp.gemm_scaled8(dmp.Scaled8(a, sa), dmp.Scaled8(b, sb, block=128), off, out=out)
    group = torch.repeat_interleave(used, rows[used]).cuda()
    want = torch.bmm(a.float()[:, None], b.view(torch.uint8)[group].view(f8).float().transpose(1, 2).contiguous())[:, 0]
    assert torch.equal(out, want)
