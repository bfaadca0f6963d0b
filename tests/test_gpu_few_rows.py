"""Grouped products of few rows (decoding), in both layouts of B: leading dimensions
larger than the rows, infinities and NaN that stay in their rows, two streams at once,
and a captured graph replayed on other offsets.  Tolerances: tests/test_gpu_grouped.py."""
import pytest

from test_gpu_grouped import bound, check, dmp, grouped_reference, normal, offsets_of  # noqa: F401

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def weights(seed, G, K, N, ld, b_col):
    """(B on the CPU, B on the GPU with leading dimension ld)."""
    B = normal(seed, G, K, N, dtype=torch.bfloat16)
    if b_col:
        big = torch.full((G, N, ld), float("nan"), dtype=torch.bfloat16, device="cuda")
        big[:, :, :K] = B.transpose(1, 2).cuda()
        return B, big[:, :, :K].transpose(1, 2)
    big = torch.full((G, K, ld), float("nan"), dtype=torch.bfloat16, device="cuda")
    big[:, :, :N] = B.cuda()
    return B, big[:, :, :N]


@pytest.mark.parametrize("b_col", [True, False], ids=["col", "row"])
@pytest.mark.parametrize("counts", [[1, 0, 3], [16, 17, 0, 1], [33, 0, 0, 0, 0, 0, 5], [2] * 300])
def test_padded_operands(dmp, counts, b_col):  # noqa: F811
    """The padding of A, B, C and D holds NaN: none is read, none is written."""
    T, K, N, off = sum(counts) + 3, 264, 136, offsets_of(counts, head=1)
    A = normal(40, T, K, dtype=torch.bfloat16)
    Ag = torch.full((T, 280), float("nan"), dtype=torch.bfloat16, device="cuda")
    Ag[:, :K] = A.cuda()
    B, Bg = weights(41, len(counts), K, N, 288, b_col)
    C = normal(42, T, N, dtype=torch.float32)
    buf = torch.full((T, 150), float("nan"), device="cuda")
    buf[:, :N] = C.cuda()
    acc, S, ref, c, owned = grouped_reference(A, B, off, 0.5, 2.0, C)
    dmp.gemm_grouped(Ag[:, :K], Bg, off.cuda(), C=buf[:, :N], out=buf[:, :N], alpha=0.5, beta=2.0)
    tol = bound(S, K, 0.5, acc, 2.0, c, ref, torch.float32)
    check(buf[:, :N][owned.cuda()], ref[owned], tol[owned], f"padded {counts[:4]}")
    assert torch.equal(buf[:, :N].cpu()[~owned], C[~owned]) and buf[:, N:].isnan().all()


@pytest.mark.parametrize("b_col", [True, False], ids=["col", "row"])
def test_not_finite_values_stay_in_their_rows_and_columns(dmp, b_col):  # noqa: F811
    counts, K, N = [3, 0, 20], 72, 136
    T, off = sum(counts), offsets_of(counts).cuda()
    A = normal(43, T, K, dtype=torch.bfloat16).cuda()
    _, B = weights(44, 3, K, N, 144, b_col)
    clean = dmp.gemm_grouped(A, B, off)
    A2, B2 = A.clone(), B.clone() if not b_col else B.transpose(1, 2).clone().transpose(1, 2)
    A2[1, K - 1], A2[5, 0] = float("nan"), float("inf")
    B2[1], B2[2, 3, 77] = float("nan"), float("nan")  # a whole group without rows; one value
    D = dmp.gemm_grouped(A2, B2, off)
    hit = torch.zeros(T, N, dtype=torch.bool, device="cuda")
    hit[1] = hit[5] = True
    hit[3:, 77] = True
    assert torch.equal(D[~hit], clean[~hit]) and not D[hit].isfinite().any()


@pytest.mark.parametrize("b_col", [True, False], ids=["col", "row"])
def test_two_streams_at_once_and_a_captured_graph(dmp, b_col):  # noqa: F811
    counts, K, N = [1, 7, 0, 16], 512, 264
    T, off = sum(counts), offsets_of(counts).cuda()
    A = normal(45, T, K, dtype=torch.bfloat16).cuda()
    _, B = weights(46, 4, K, N, K if b_col else N, b_col)
    want = dmp.gemm_grouped(A, B, off)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.zeros(20, T, N, device="cuda") for _ in streams]
    torch.cuda.synchronize()
    for i in range(20):
        for s, o in zip(streams, outs):
            with torch.cuda.stream(s):
                dmp.gemm_grouped(A, B, off, out=o[i])
    torch.cuda.synchronize()
    assert all((o == want).all() for o in outs)

    out = torch.zeros(T, N, device="cuda")
    graph, s = torch.cuda.CUDAGraph(), streams[0]
    with torch.cuda.stream(s):
        dmp.gemm_grouped(A, B, off, out=out)
        s.synchronize()
        with torch.cuda.graph(graph, stream=s):
            dmp.gemm_grouped(A, B, off, out=out)
    for other in ([1, 7, 0, 16], [0, 0, 24, 0], [24, 0, 0, 0], [6, 6, 6, 6]):
        off.copy_(offsets_of(other))
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, dmp.gemm_grouped(A, B, off)), other
