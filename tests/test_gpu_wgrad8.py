"""Weight gradients from 8-bit checkpoints (gemm_wgrad8) and quantization with powers of
two as scales (quant8's pow2) on the GPU against a plain 64-bit computation on the CPU.

Tolerance per element, from the arithmetic alone.  With x = q * s rounded to Y's type as
the definition says (exact for powers of two), the bound of the 16-bit gradients: 4 K u of
the sum of magnitudes (u = 2^-24, K the group's rows; splitting the rows adds no more
roundings than the sum has), three roundings of the output stage, half a step of the
output type.  Rounding q * s first in 32 bits and then to 16 is off from rounding once by
at most a step's tie, one step of 32 bits in the product: u of the magnitudes more."""
import numpy as np
import pytest

from gpu_util import log

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
Q = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
U = 2.0 ** -24


@pytest.fixture(scope="module")
def dmp():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import dense_mixed_precision_02_amd as dmp
    return dmp


def normal(seed, *shape, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype)


def pow2_reference(x, q):
    """(values q as float64, scales) of the definition, in 64 bits on the CPU."""
    rows, m = x.shape
    top = 448.0 if q == "e4m3" else 57344.0
    kb = -(-m // 128)
    v = torch.nn.functional.pad(x.double(), (0, kb * 128 - m)).reshape(rows, kb, 128)
    a = v.abs().amax(-1).clamp_min(2.0 ** -100)
    s = torch.exp2(torch.ceil(torch.log2(a / top)))
    s = torch.where(s / 2 * top >= a, s / 2, s)  # whatever log2 rounds
    s = torch.where(s * top < a, s * 2, s)
    # the largest number of x's type with the 8-bit type's digits
    end = 2.0 ** (15 if x.dtype == torch.float16 else 127) * (1.875 if q == "e4m3" else 1.75)
    v = v.clamp(-end, end)
    v = v / s[..., None]
    mant, low = (3, -6) if q == "e4m3" else (2, -14)
    place = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** low))) - mant)
    return (torch.round(v / place) * place).reshape(rows, kb * 128)[:, :m], s


@pytest.mark.parametrize("q", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_pow2_scales(dmp, q, dtype):
    top = 448.0 if q == "e4m3" else 57344.0
    for m in (1, 16, 100, 128, 129, 1000, 1024):
        x = normal(m, 37, m) * torch.exp2(torch.randint(-30, 10, (37, 1), generator=torch.Generator().manual_seed(1)).float())
        x[3] = 0
        x[4] = 2.0 ** -14
        x[5, 0] = 448.0 if dtype == "f16" else top * 4  # at the border of two scales
        x[6, -1] = -448.0 * 1.01
        x = x.to(DT[dtype])
        x[7] = torch.finfo(DT[dtype]).max
        want, scale = pow2_reference(x, q)
        r = dmp.quant8(x.cuda(), dtype=Q[q], pow2=True)
        assert torch.equal(r.scale.cpu().double(), scale)
        got = r.q.cpu().double()
        assert torch.equal(got[:, :m], want) and not got[:, m:].any()
        # what the operand stands for is a number of 16 bits
        value = got[:, :m] * scale.repeat_interleave(128, 1)[:, :m]
        t = torch.float16 if dtype == "f16" else torch.bfloat16
        assert torch.equal(value.to(t).double(), value)


def test_pow2_of_other_layouts_and_blocks(dmp):
    x = normal(1, 300, 200, dtype=torch.bfloat16)
    want, scale = pow2_reference(x, "e4m3")
    r = dmp.quant8(x.t().contiguous().cuda().t(), pow2=True)
    assert torch.equal(r.q.cpu().double()[:, :200], want) and torch.equal(r.scale.cpu().double(), scale)
    r = dmp.quant8(x.cuda(), block=128, pow2=True)
    s = torch.stack([scale[i:i + 128].amax(0) for i in range(0, 300, 128)])  # monotonic in the maximum
    assert torch.equal(r.scale.cpu().double(), s)
    x[5, 7] = float("inf")
    r = dmp.quant8(x.cuda(), pow2=True)
    assert r.scale[5, 0].isnan() and not r.scale[5, 1].isnan() and not r.q.float()[5, :128].any()
    a, b = dmp.quant8(x.cuda()), dmp.quant8(x.cuda(), pow2=False)
    assert torch.equal(a.q.view(torch.uint8), b.q.view(torch.uint8))


def operand(dmp, seed, T, M, q, pow2=True):
    """An operand and the values it stands for (float64)."""
    kp, kb = -(-M // 16) * 16, -(-M // 128)
    x = normal(seed, T, kp)
    x[:, M:] = 0
    q8 = (x * (20.0 if q == "e4m3" else 2000.0)).to(Q[q])
    s = torch.exp2(torch.randint(-8, 3, (T, kb), generator=torch.Generator().manual_seed(seed)).float())
    if not pow2:
        s = s * (1 + torch.rand(T, kb, generator=torch.Generator().manual_seed(seed + 1)))
    return q8, s


def reference(q8, s, Y, M, off, alpha, beta, C):
    """(sum, magnitudes, result) group by group in 64 bits, x rounded to Y's type."""
    x = (q8[:, :M].double() * s.double().repeat_interleave(128, 1)[:, :M]).to(Y.dtype).double()
    y = Y.double()
    acc = torch.stack([x[a:b].t() @ y[a:b] for a, b in zip(off[:-1], off[1:])])
    S = torch.stack([x[a:b].abs().t() @ y[a:b].abs() for a, b in zip(off[:-1], off[1:])])
    c = C.double() if C is not None else torch.zeros_like(acc)
    return acc, S, alpha * acc + beta * c, c


def check(got, acc, S, want, c, rows, alpha, beta):
    got = got.double().cpu().reshape(want.shape)
    low = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}
    t = check.type
    tol = (4.0 * rows + 1) * U * abs(alpha) * S * 1.01 + U * (abs(alpha) * acc.abs() + (beta * c).abs() + 2 * want.abs()) * 1.01 \
        + torch.finfo(t).eps / 2 * want.abs() * 1.01 + low[t]
    # values beyond Y's type (fp16: e5m2 times a factor) are infinities by the definition, in the sums too
    end = ~torch.isfinite(want)
    assert torch.equal(torch.nan_to_num(got[end], nan=1.0), torch.nan_to_num(want[end], nan=1.0))
    got, want, tol = got[~end], want[~end], tol[~end]
    assert torch.isfinite(got).all()
    bad = (got - want).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} over the bound, worst {float(((got - want).abs() / tol).max()):.3g}"


# Y's type, q, counts of the groups (None: one group of all rows), head, tail, M, N, out, alpha, beta
CASES = [
    ("bf16", "e4m3", None, 1, 0, 1, 1, "f32", 1.0, 0.0),
    ("f16", "e4m3", None, 0, 0, 8, 8, "f32", 1.0, 0.0),       # no rows
    ("bf16", "e5m2", None, 64, 0, 64, 128, "bf16", 1.0, 0.0),
    ("f16", "e4m3", None, 65, 0, 130, 136, "f16", 0.5, 2.0),
    ("bf16", "e4m3", None, 1000, 0, 72, 40, "f32", 1.0, 1.0),   # rows split
    ("bf16", "e4m3", None, 3001, 0, 130, 99, "bf16", 1.0, 0.5),  # the same, unaligned
    ("f16", "e5m2", None, 5000, 0, 17, 264, "f32", 2.0, 0.0),
    ("bf16", "e4m3", [0, 5, 64, 0, 65, 1, 0], 3, 9, 136, 200, "f32", 1.0, 1.0),
    ("f16", "e4m3", [17, 0, 129], 0, 5, 99, 33, "f16", 1.0, 0.0),
    ("bf16", "e5m2", [700, 0, 1, 900], 2, 3, 200, 72, "bf16", 1.0, 1.0),
    ("f16", "e4m3", [2000, 0, 1, 3001], 2, 3, 200, 72, "f32", 1.0, 1.0),  # groups whose rows are split
    ("bf16", "e4m3", [3, 0, 70, 1] * 20, 0, 0, 64, 128, "f32", 1.0, 0.0),  # more than 64 groups
    ("bf16", "e4m3", None, 520, 0, 4096, 4096, "bf16", 1.0, 0.0),  # 256 x 256 tiles
    ("f16", "e5m2", [1030, 0, 864, 361], 5, 6, 2000, 2200, "f32", 0.5, 1.0),  # the same, partial tiles
    ("bf16", "e4m3", None, 4099, 0, 2000, 1999, "bf16", 1.0, 1.0),  # the same, rows split, unaligned
    ("f16", "e4m3", [1500, 700, 0], 1, 2, 1000, 1400, "f16", 1.0, 0.0),  # 128 x 128 tiles
    ("bf16", "e5m2", None, 5003, 0, 900, 650, "f32", 1.0, 0.5),  # the same, rows split
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}-{c[1]}-g{len(c[2]) if c[2] else 0}-{c[3]}-{c[5]}x{c[6]}-{c[7]}")
@pytest.mark.parametrize("pow2", [True, False])
def test_wgrad8(dmp, case, pow2):
    dt, q, counts, head, tail, M, N, out, alpha, beta = case
    log(f"[wgrad8] {case} {pow2}")
    T = head + sum(counts) + tail if counts is not None else head
    off = [0, T] if counts is None else [head] + [int(v) for v in head + np.cumsum(counts)]
    q8, s = operand(dmp, 1, T, M, q, pow2)
    Y = normal(2, T, N, dtype=DT[dt])
    shape = (len(off) - 1, M, N) if counts is not None else (M, N)
    C = normal(3, *shape, dtype=DT[out]) if beta else None
    acc, S, want, c = reference(q8, s, Y, M, off, alpha, beta, C.reshape(-1, M, N) if beta else None)
    X = dmp.Scaled8(q8.cuda(), s.cuda(), K=M)
    offsets = torch.tensor(off).cuda() if counts is not None else None
    D = torch.full(shape, 7.0, dtype=DT[out], device="cuda")
    r = dmp.gemm_wgrad8(X, Y.cuda(), offsets, C.cuda() if beta else None, out=D, alpha=alpha, beta=beta)
    assert r is D
    check.type = DT[out]
    check(D, acc, S, want, c, max(b - a for a, b in zip(off[:-1], off[1:])), alpha, beta)
    D2 = dmp.gemm_wgrad8(X, Y.cuda(), offsets.int() if offsets is not None else None, C.cuda() if beta else None,
                         alpha=alpha, beta=beta, out_dtype=DT[out])
    assert torch.equal(D, D2)


def test_steps_of_a_layer(dmp):
    """A layer's input kept in 8 bits and its weight gradient from that, next to the gradient from
    the input itself: the same sums of the rounded values."""
    T, M, N = 700, 264, 136
    x, dy = normal(1, T, M, dtype=torch.bfloat16).cuda(), normal(2, T, N, dtype=torch.bfloat16).cuda()
    off = torch.tensor([0, 300, 300, 700], device="cuda")
    kept = dmp.quant8(x, pow2=True)
    value = (kept.q[:, :M].float() * kept.scale.repeat_interleave(128, 1)[:, :M]).bfloat16()
    got, want = dmp.gemm_wgrad8(kept, dy, off), dmp.gemm_grouped_wgrad(value, dy, off)
    S = dmp.gemm_grouped_wgrad(value.abs(), dy.abs(), off)
    # both lie within 4 K u of the exact sum
    assert ((got - want).abs() <= 2 * 4 * 400 * U * S * 1.01).all()
    # and the checkpoint's own error: half a step of 4 bits for every value (2^-4 of it, or of
    # the least normal, 2^-6 scales)
    exact = dmp.gemm_grouped_wgrad(x, dy, off)
    step = (x.float().abs() * 2.0 ** -4).clamp_min(2.0 ** -10 * float(kept.scale.max())).bfloat16()
    assert ((got - exact).abs() <= dmp.gemm_grouped_wgrad(step, dy.abs(), off) * 1.02 + 1e-3).all()


def test_what_is_no_number_shows(dmp):
    q8, s = operand(dmp, 1, 100, 300, "e4m3")
    s[50, 1] = float("nan")
    Y = normal(2, 100, 64, dtype=torch.bfloat16).cuda()
    D = dmp.gemm_wgrad8(dmp.Scaled8(q8.cuda(), s.cuda(), K=300), Y)
    assert D[128:256].isnan().all() and torch.isfinite(D[:128]).all() and torch.isfinite(D[256:]).all()
    # rows that no group owns are not read: their NaN does not show
    off = torch.tensor([0, 50], device="cuda")
    assert torch.isfinite(dmp.gemm_wgrad8(dmp.Scaled8(q8.cuda(), s.cuda(), K=300), Y, off)).all()
    off = torch.tensor([51, 100], device="cuda")
    assert torch.isfinite(dmp.gemm_wgrad8(dmp.Scaled8(q8.cuda(), s.cuda(), K=300), Y, off)).all()


def test_strides_and_views(dmp):
    """Rows of q, Y and D further apart than their widths, scales of both orders, D over C."""
    q8, s = operand(dmp, 5, 600, 200, "e4m3")
    wide = torch.zeros(600, 256, dtype=torch.uint8).view(Q["e4m3"]).cuda()
    wide.view(torch.uint8)[:, 16:16 + 208] = q8.cuda().view(torch.uint8)
    Yw = normal(6, 600, 200, dtype=torch.bfloat16).cuda()
    Y = Yw[:, 8:144]
    plain = dmp.gemm_wgrad8(dmp.Scaled8(q8.cuda(), s.cuda(), K=200), Y.contiguous())
    X = dmp.Scaled8(wide[:, 16:224], s.cuda().t().contiguous().t(), K=200)
    D = torch.full((200, 300), 7.0, device="cuda")
    dmp.gemm_wgrad8(X, Y, out=D[:, 100:236])
    assert torch.equal(D[:, 100:236], plain) and (D[:, :100] == 7).all() and (D[:, 236:] == 7).all()
    C = normal(7, 200, 136).cuda()
    want = dmp.gemm_wgrad8(X, Y, None, C)
    assert dmp.gemm_wgrad8(X, Y, None, C, out=C) is C and torch.equal(C, want)


def test_streams_and_captured_graphs(dmp):
    """Split sums need scratch: each call has its own, on two streams and in two graphs that are
    replayed in turn."""
    ops = [(operand(dmp, 10 + i, 4000, 128, "e4m3"), normal(20 + i, 4000, 128, dtype=torch.bfloat16).cuda()) for i in range(2)]
    X = [dmp.Scaled8(q.cuda(), s.cuda(), K=128) for (q, s), _ in ops]
    Y = [y for _, y in ops]
    want = [dmp.gemm_wgrad8(x, y) for x, y in zip(X, Y)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(8):
        with torch.cuda.stream(streams[i % 2]):
            got.append(dmp.gemm_wgrad8(X[i % 2], Y[i % 2]))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i % 2]) for i, g in enumerate(got))
    graphs, outs = [], []
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(dmp.gemm_wgrad8(X[i], Y[i]))
        graphs.append(graph)
    for i in range(6):
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i % 2], want[i % 2])
        Y[i % 2].mul_(2.0)
        want[i % 2] = dmp.gemm_wgrad8(X[i % 2], Y[i % 2])
        torch.cuda.synchronize()
