"""8-bit quantization (quant8) and the 8-bit block-scaled products (gemm_scaled8) on
the GPU.  quant8 is compared bit for bit with the same fp32 steps on the CPU; the
product with a 64-bit computation on the same 8-bit values and scales.

Tolerance of the product per element: the header's 4 (K + 128) 2^-24 S (S: the sum of
the scaled products' magnitudes), three fp32 roundings of the output stage, half a
step of the output type."""
import numpy as np
import pytest

from gpu_util import log

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
TOP = {E4: 448.0, E5: 57344.0}
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def dmp():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import dense_mixed_precision_02_amd as dmp
    return dmp


def normal(seed, *shape, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype)


def offsets_of(counts, head=0):
    return torch.tensor([head] + [int(x) for x in head + np.cumsum(counts)], dtype=torch.int64)


def quant_reference(X, block, dtype):
    """(q as 8-bit floats, scale), the definition's fp32 steps one by one on the CPU."""
    x = X.float().numpy()
    top = np.float32(TOP[dtype])
    *lead, M, K = x.shape
    kb, mb = -(-K // 128), -(-M // block)
    x = x.reshape(-1, M, K)
    v = np.zeros_like(x)
    scale = np.zeros((x.shape[0], mb, kb), dtype=np.float32)
    with np.errstate(all="ignore"):
        for b in range(x.shape[0]):
            for i in range(mb):
                for k in range(kb):
                    s = np.s_[b, i * block:(i + 1) * block, k * 128:(k + 1) * 128]
                    a = np.abs(x[s]).max()
                    if not np.isfinite(x[s]).all():
                        scale[b, i, k] = np.nan
                        continue
                    a = max(np.float32(a), np.float32(2.0 ** -100))
                    scale[b, i, k] = a / top
                    v[s] = x[s] * (top / a)
    return torch.from_numpy(v.reshape(*lead, M, K)).to(dtype), torch.from_numpy(scale.reshape(*lead, mb, kb))


# shape, dtype of X, transposed
QUANT = [
    ((1, 1), "f32", False), ((1, 4096), "bf16", False), ((3, 130), "f16", False), ((17, 1000), "bf16", False),
    ((129, 257), "f32", False), ((64, 1031), "f16", False), ((300, 128), "bf16", False),
    ((2, 70, 200), "bf16", False), ((3, 129, 130), "f32", False),
    ((1, 1), "f32", True), ((5, 300), "bf16", True), ((130, 64), "f16", True), ((257, 129), "f32", True),
    ((2, 200, 140), "bf16", True), ((128, 512), "bf16", True), ((1000, 17), "f16", True),
]


@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("fmt", [E4, E5], ids=["e4m3", "e5m2"])
@pytest.mark.parametrize("case", QUANT, ids=lambda c: f"{'x'.join(map(str, c[0]))}-{c[1]}{'-t' if c[2] else ''}")
def test_quant8_bit_for_bit(dmp, case, fmt, block):
    shape, dt, tr = case
    X = normal(1, *shape) * torch.exp(3 * normal(2, *shape[:-1], 1))
    X = X.to(DT[dt])
    X[..., -1, :] = 0 if shape[-2] > 2 else X[..., -1, :]  # a row of zeros
    Xd = X.transpose(-1, -2).contiguous().cuda().transpose(-1, -2) if tr else X.cuda()
    log(f"[quant8] {case} {fmt} block {block}")
    r = dmp.quant8(Xd, block=block, dtype=fmt)
    q, scale = quant_reference(X, block, fmt)
    K = shape[-1]
    assert r.q.shape[-1] == -(-K // 16) * 16 and r.q.dtype == fmt
    assert torch.equal(r.q[..., :K].cpu().view(torch.uint8), q.view(torch.uint8))
    assert (r.q[..., K:].cpu().view(torch.uint8) == 0).all()
    assert torch.equal(r.scale.cpu(), scale)


@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("tr", [False, True], ids=["rows", "transposed"])
def test_quant8_values_at_the_border(dmp, block, tr):
    """Infinities, NaN, the largest floats, subnormals and zeros: such blocks get the
    scale NaN and zeros, or the least scale; the blocks beside them are not touched."""
    X = normal(3, 256, 256)
    X[0, 0], X[1, 130], X[129, 255] = float("inf"), float("nan"), float("-inf")
    X[5, :128] = 2.0 ** -140
    X[6, 128:] = 0.0
    X[130, :128] *= 1e38
    Xd = X.t().contiguous().cuda().t() if tr else X.cuda()
    r = dmp.quant8(Xd, block=block)
    q, scale = quant_reference(X, block, E4)
    assert torch.equal(r.q.cpu().view(torch.uint8), q.view(torch.uint8))
    assert torch.equal(torch.isnan(r.scale.cpu()), torch.isnan(scale))
    assert torch.equal(torch.nan_to_num(r.scale.cpu()), torch.nan_to_num(scale))


def test_quant8_strided_and_unaligned(dmp):
    buf = normal(4, 40 * 300 + 1).to(torch.bfloat16).cuda()
    for X in (buf[1:].view(40, 300)[:, :200], buf[:-1].view(40, 300)[:, 3:203], buf[1:].view(40, 300)[:, 5:100].t()):
        for block in (1, 128):
            r = dmp.quant8(X, block=block)
            q, scale = quant_reference(X.cpu(), block, E4)
            assert torch.equal(r.q[..., :X.shape[-1]].cpu().view(torch.uint8), q.view(torch.uint8))
            assert torch.equal(r.scale.cpu(), scale)


def values(o, K):
    """What an 8-bit operand stands for, in 64 bits."""
    rows = o.q.shape[-2]
    s = o.scale.double().cpu().repeat_interleave(128, -1)[..., :K]
    if o.block > 1:
        s = s.repeat_interleave(o.block, -2)[..., :rows, :]
    return o.q[..., :K].double().cpu() * s


def make8(dmp, seed, lead, rows, K, fmt, block):
    """Random 8-bit values (zeros and the largest among them) with scales over powers of
    two, in a [k-block][row] table."""
    kp = -(-K // 16) * 16
    x = (normal(seed, *lead, rows, kp) * (TOP[fmt] / 4)).clamp(-TOP[fmt], TOP[fmt])
    x[..., K:] = 0
    scale = torch.exp2(2 * normal(seed + 1, *lead, -(-K // 128), -(-rows // block))) / TOP[fmt]
    return dmp.Scaled8(x.to(fmt).cuda(), scale.cuda().transpose(-1, -2), block=block, K=K)


def check(got, A, B, off, alpha, beta, C, out_dtype, K):
    a, b = values(A, K), values(B, K)
    off = [0, a.shape[0]] if off is None else [int(x) for x in off]
    b = b[None] if b.dim() == 2 else b
    got = got.double().cpu()
    u = 2.0 ** -24
    for g in range(len(off) - 1):
        s = slice(off[g], off[g + 1])
        acc, S = a[s] @ b[g].t(), a[s].abs() @ b[g].abs().t()
        c = C[s].double().cpu() if C is not None else torch.zeros_like(acc)
        ref = alpha * acc + beta * c
        tol = 4 * (K + 128) * u * abs(alpha) * S * 1.01 + u * 1.01 * (abs(alpha) * acc.abs() + (beta * c).abs() + 2 * ref.abs()) + \
            torch.finfo(out_dtype).eps / 2 * ref.abs() * 1.01 + 2.0 ** -25
        assert torch.isfinite(got[s]).all()
        bad = (got[s] - ref).abs() > tol
        assert not bad.any(), f"group {g}: {int(bad.sum())} over the bound, worst " \
            f"{float(((got[s] - ref).abs() / tol).max()):.3g}"


# T or counts, K, N, format of A, of B, out, alpha, beta
SCALED = [
    (1, 16, 1, E4, E4, "f32", 1.0, 0.0), (1, 1, 1, E4, E5, "f32", 1.0, 0.0), (1, 4096, 512, E4, E4, "bf16", 1.0, 0.0),
    (16, 2048, 300, E4, E4, "f16", 0.001, 0.0), (40, 130, 129, E5, E4, "f32", 1.0, 0.0),
    (130, 384, 256, E4, E5, "f32", 0.5, 2.0), (257, 1040, 385, E5, E5, "f32", 1.0, 1.0),
    (512, 512, 512, E4, E4, "bf16", 1.0, 0.0), (300, 127, 640, E4, E4, "f32", 1.0, 0.0),
    (1025, 640, 520, E4, E4, "f32", 1.0, 0.0),
    ([1, 0, 2], 256, 128, E4, E4, "f32", 1.0, 0.0), ([64, 0, 65, 1, 200], 400, 264, E5, E4, "bf16", 1.0, 1.0),
    ([300, 257, 0, 511], 512, 384, E4, E4, "f32", 1.0, 0.0), ([1] * 70 + [0, 5], 144, 72, E4, E4, "f32", 1.0, 0.0),
    ([17, 40, 3], 2064, 200, E4, E5, "f32", 1.0, 0.0),
    # few rows to a group, 32 and 64 columns to a workgroup, one group with many
    ([1, 2, 0, 5] * 25, 272, 72, E4, E4, "bf16", 1.0, 1.0), ([70] + [0] * 150 + [1] * 50, 272, 72, E5, E4, "f32", 1.0, 0.0),
]


@pytest.mark.parametrize("case", SCALED, ids=lambda c: f"{c[0] if isinstance(c[0], int) else 'g%d' % len(c[0])}-{c[1]}x{c[2]}")
def test_scaled8(dmp, case):
    rows, K, N, fa, fb, out, alpha, beta = case
    log(f"[scaled8] {case}")
    grouped = not isinstance(rows, int)
    T = sum(rows) + 12 if grouped else rows
    off = offsets_of(rows, 5) if grouped else None
    A = make8(dmp, 10, (), T, K, fa, 1)
    B = make8(dmp, 20, (len(rows),) if grouped else (), N, K, fb, 128)
    C = normal(30, T, N).to(DT[out]).cuda() if beta else None
    D = torch.full((T, N), 7.0, dtype=DT[out], device="cuda")
    dmp.gemm_scaled8(A, B, off.cuda() if grouped else None, C, out=D, alpha=alpha, beta=beta)
    check(D, A, B, off, alpha, beta, C, DT[out], K)
    if grouped:
        assert (D[:5] == 7.0).all() and (D[T - 7:] == 7.0).all()
        E = torch.full((T, N), 7.0, dtype=DT[out], device="cuda")
        dmp.gemm_scaled8(A, B, off.int().cuda(), C, out=E, alpha=alpha, beta=beta)
        assert torch.equal(D, E)
    # the scales' strides are free: the same from [row][k-block] tables
    A2 = dmp.Scaled8(A.q, A.scale.contiguous(), block=1, K=K)
    B2 = dmp.Scaled8(B.q, B.scale.contiguous(), block=128, K=K)
    F = torch.full((T, N), 7.0, dtype=DT[out], device="cuda")
    dmp.gemm_scaled8(A2, B2, off.cuda() if grouped else None, C, out=F, alpha=alpha, beta=beta)
    assert torch.equal(D, F)


@pytest.mark.parametrize("fa,fb", [(E4, E4), (E5, E4), (E4, E5), (E5, E5)])
@pytest.mark.parametrize("T,K,N", [(5, 256, 200), (260, 384, 264), (600, 1024, 512)])
def test_small_integers_are_exact(dmp, fa, fb, T, K, N):
    """Integers up to 4 with power-of-two scales: every product and sum is exact."""
    g = torch.Generator().manual_seed(5)
    a, b = torch.randint(-4, 5, (T, K), generator=g).float(), torch.randint(-4, 5, (N, K), generator=g).float()
    sa = torch.exp2(torch.randint(-2, 3, (T, K // 128), generator=g).float())
    sb = torch.exp2(torch.randint(-2, 3, (-(-N // 128), K // 128), generator=g).float())
    A, B = dmp.Scaled8(a.to(fa).cuda(), sa.cuda()), dmp.Scaled8(b.to(fb).cuda(), sb.cuda(), block=128)
    D = dmp.gemm_scaled8(A, B)
    assert torch.equal(D.double().cpu(), values(A, K) @ values(B, K).t())


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("counts", [None, [1700, 0, 1501, 1200]], ids=["dense", "grouped"])
def test_largest_tiles_small_integers(dmp, counts, out):
    """Enough tiles for the largest kernels; integers whose sums stay below 2^8 (bf16) or
    2^24 in magnitude: exact."""
    K, N, T = 272, 4000, 4410
    g = torch.Generator(device="cuda").manual_seed(6)
    G = 1 if counts is None else len(counts)
    density = 0.02 if out == "bf16" else 1.0  # about 5 products of at most 16 to a sum
    a = torch.randint(-4, 5, (T, K), generator=g, device="cuda").float()
    b = torch.randint(-4, 5, (G, N, K), generator=g, device="cuda").float()
    a = a * (torch.rand(T, K, generator=g, device="cuda") < density)
    B = dmp.Scaled8((b if counts else b[0]).to(E5), torch.full((G, 32, 3) if counts else (32, 3), 2.0, device="cuda"),
                    block=128)
    A = dmp.Scaled8(a.to(E4), torch.full((T, 3), 0.5, device="cuda"))
    off = None if counts is None else offsets_of(counts, 4)
    D = torch.full((T, N), 7.0, device="cuda").to(DT[out])
    dmp.gemm_scaled8(A, B, off.cuda() if counts else None, out=D)
    want = torch.full((T, N), 7.0, device="cuda", dtype=torch.float64)
    for i in range(G):
        s = slice(int(off[i]), int(off[i + 1])) if counts else slice(0, T)
        want[s] = a[s].double() @ b[i].double().t().contiguous()
    keep = want.abs() <= (256 if out == "bf16" else 1 << 24)
    assert keep.double().mean() > 0.99
    assert torch.equal(D.double()[keep], want[keep])


def test_not_finite_scale_reaches_its_rows_and_columns_only(dmp):
    A, B = make8(dmp, 40, (), 200, 256, E4, 1), make8(dmp, 50, (), 300, 256, E4, 128)
    clean = dmp.gemm_scaled8(A, B)
    A.scale[7, 1] = float("nan")
    D = dmp.gemm_scaled8(A, B)
    assert torch.isnan(D[7]).all()
    keep = [i for i in range(200) if i != 7]
    assert torch.equal(D[keep], clean[keep])
    A.scale[7, 1] = 1.0
    B.scale[1, 0] = float("nan")
    D = dmp.gemm_scaled8(A, B)
    assert torch.isnan(D[:, 128:256]).all()
    assert torch.equal(D[keep][:, :128], clean[keep][:, :128]) and torch.equal(D[keep][:, 256:], clean[keep][:, 256:])


def test_k0_and_empty(dmp):
    A = dmp.quant8(torch.empty(3, 0, device="cuda"))
    B = dmp.quant8(torch.empty(8, 0, device="cuda"), block=128)
    C = torch.arange(24.0, device="cuda").view(3, 8)
    assert torch.equal(dmp.gemm_scaled8(A, B, None, C, beta=0.5), 0.5 * C)
    A = dmp.quant8(torch.empty(0, 32, device="cuda"))
    B = dmp.quant8(torch.ones(8, 32, device="cuda"), block=128)
    assert dmp.gemm_scaled8(A, B).shape == (0, 8)


def test_quantized_expert_layer_as_used(dmp):
    """An expert block in 8 bits as serving runs it: tokens quantized by rows, weights
    (stored K x N) once by blocks; products, activation, quantization, product.  Each
    operator is compared with the 64-bit result on the operands that it was given, and
    the whole with the unquantized block: two quantizations (each value off by half a
    step, 2^-4 relative or 2^-10 of the block's largest, which is at most about 5
    deviations) on either side of two products leave errors that average out over K;
    0.1 of the result's norm bounds four independent relative errors of 2^-4 / sqrt(3)
    (uniform in the step) with margin: sqrt(4) * 2^-4 / sqrt(3) = 0.072."""
    counts, K, H = [40, 0, 3, 85], 256, 384
    T, G, off = sum(counts), len(counts), offsets_of(counts)
    X = normal(60, T, K, dtype=torch.bfloat16).cuda()
    W1 = (normal(61, G, K, H) / 16).to(torch.bfloat16).cuda()
    W2 = (normal(62, G, H, K) / 20).to(torch.bfloat16).cuda()
    W1q, W2q = dmp.quant8(W1.transpose(1, 2), block=128), dmp.quant8(W2.transpose(1, 2), block=128)
    Xq = dmp.quant8(X)
    h = dmp.gemm_scaled8(Xq, W1q, off.cuda(), out_dtype=torch.bfloat16)
    check(h, Xq, W1q, off, 1.0, 0.0, None, torch.bfloat16, K)
    aq = dmp.quant8(torch.nn.functional.silu(h.float()).to(torch.bfloat16))
    y = dmp.gemm_scaled8(aq, W2q, off.cuda())
    check(y, aq, W2q, off, 1.0, 0.0, None, torch.float32, H)
    full = dmp.gemm_grouped(torch.nn.functional.silu(dmp.gemm_grouped(X, W1, off.cuda())).to(torch.bfloat16), W2, off.cuda())
    assert float((y - full).norm() / full.norm()) < 0.1


def test_captured_graph_and_other_stream(dmp):
    T, K, N, G = 150, 256, 264, 3
    X, W = normal(70, T, K, dtype=torch.bfloat16).cuda(), normal(71, G, N, K, dtype=torch.bfloat16).cuda()
    off = offsets_of([100, 0, 50]).cuda()
    B = dmp.quant8(W, block=128)
    out = torch.zeros(T, N, device="cuda")
    want = dmp.gemm_scaled8(dmp.quant8(X), B, off)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        dmp.gemm_scaled8(dmp.quant8(X), B, off, out=out)
    s.synchronize()
    assert torch.equal(out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        dmp.gemm_scaled8(dmp.quant8(X), B, off, out=out)
    for r in range(3):
        out.zero_()
        dmp.gemm_scaled8(dmp.quant8(X), B, off)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), f"replay {r}"
    X.copy_(normal(72, T, K, dtype=torch.bfloat16))
    off.copy_(offsets_of([1, 2, 147]))
    want = dmp.gemm_scaled8(dmp.quant8(X), B, off)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
