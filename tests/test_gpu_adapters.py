"""Low-rank adapters beside a shared projection (gemm_adapters) on the GPU against a plain
64-bit computation on the CPU.

Tolerance per element, from the arithmetic alone (u = 2^-24).  A hidden value h = s * sum x a:
4 K u |s| S_h for the sum (S_h: of magnitudes), 2 u |h| for the waves' join and the scale, and
its rounding to 16 bits: half a step, e |h| with e = 2^-8 (bf16) or 2^-11 (fp16), and half of
fp16's least subnormal, 2^-25; where D is fp32 the rest of that is kept too: e^2 |h| for fp16, and again 2^-25; e^3 |h| for bf16.
The product: 4 (K + n r) u (S_w + sum |h b|), n the parts of h, and the hidden values' errors times
|b|; then the output stage's three roundings and half a step of the output type."""
import numpy as np
import pytest

from gpu_util import log

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
U = 2.0 ** -24
E16 = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(scope="module")
def dmp():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import dense_mixed_precision_02_amd as dmp
    return dmp


def normal(seed, *shape, dtype=torch.float32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def operands(seed, T, K, N, r, a, dtype, linear):
    """X, W, A, B on the CPU; linear: transposed views of linear layers' (outputs by inputs)."""
    X = normal(seed, T, K, dtype=dtype)
    sk = 1 / max(1.0, K ** 0.5)
    if linear:
        return (X, normal(seed + 1, N, K, dtype=dtype, scale=sk).t(), normal(seed + 2, a, r, K, dtype=dtype, scale=sk).transpose(1, 2),
                normal(seed + 3, a, N, r, dtype=dtype).transpose(1, 2))
    return (X, normal(seed + 1, K, N, dtype=dtype, scale=sk), normal(seed + 2, a, K, r, dtype=dtype, scale=sk),
            normal(seed + 3, a, r, N, dtype=dtype))


def to_gpu(x):
    """The same view on the GPU (contiguous storage, same strides)."""
    if x.dim() >= 2 and x.stride(-1) != 1:
        return x.transpose(-1, -2).contiguous().cuda().transpose(-1, -2)
    return x.contiguous().cuda()


def reference(X, W, A, B, off, ids, scale, alpha, beta, C, out_dtype):
    """(result, tolerance, hidden, its tolerance, owned rows) in 64 bits."""
    T, K, N, r = X.shape[0], X.shape[1], W.shape[1], A.shape[2]
    e, parts = E16[X.dtype], 1 if out_dtype != torch.float32 else 2 if X.dtype == torch.float16 else 3
    x, w = X.double(), W.double()
    acc, size, err = x @ w, x.abs() @ w.abs(), torch.zeros(T, N, dtype=torch.float64)
    h, htol = torch.zeros(T, r, dtype=torch.float64), torch.zeros(T, r, dtype=torch.float64)
    owned = torch.zeros(T, dtype=torch.bool)
    least = 2.0 ** -25 if X.dtype == torch.float16 else 2.0 ** -134
    for g in range(len(off) - 1):
        lo, hi = int(off[g]), int(off[g + 1])
        owned[lo:hi] = True
        a = int(ids[g]) if ids is not None else g
        if not 0 <= a < A.shape[0] or lo >= hi:
            continue
        s = float(scale[a]) if scale is not None else 1.0
        Aa, Ba = A[a].double(), B[a].double()
        h[lo:hi] = s * (x[lo:hi] @ Aa)
        S = abs(s) * (x[lo:hi].abs() @ Aa.abs())
        base = 4 * K * U * S + 2 * U * h[lo:hi].abs()
        htol[lo:hi] = base + e * h[lo:hi].abs() * 1.01 + least
        used = htol[lo:hi] if parts == 1 else base + e ** parts * h[lo:hi].abs() * 1.01 + least
        acc[lo:hi] += h[lo:hi] @ Ba
        size[lo:hi] += h[lo:hi].abs() @ Ba.abs()
        err[lo:hi] = used @ Ba.abs()
    c = C.double() if C is not None else torch.zeros_like(acc)
    want = alpha * acc + beta * c
    low = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}[out_dtype]
    tol = abs(alpha) * (4 * (K + parts * r) * U * size * 1.02 + err * 1.02) + \
        U * (abs(alpha) * acc.abs() + (beta * c).abs() + 2 * want.abs()) * 1.01 + \
        torch.finfo(out_dtype).eps / 2 * want.abs() * 1.01 + low
    return want, tol, h, htol, owned


def close(got, want, tol, what):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), what
    bad = (got - want).abs() > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} over the bound, worst {float(((got - want).abs() / tol).max()):.3g}"


# dtype, rows of the requests, head, tail, adapters, ids (None, or numbers), K, N, r, linear, out, alpha, beta
CASES = [
    ("f16", [1], 0, 0, 1, None, 1, 1, 1, True, "f32", 1.0, 0.0),
    ("bf16", [1], 0, 0, 1, None, 64, 64, 8, False, "bf16", 1.0, 0.0),
    ("bf16", [1, 1, 1, 1], 0, 0, 3, [0, 2, -1, 0], 512, 512, 8, True, "bf16", 1.0, 0.0),
    ("f16", [1] * 64, 0, 0, 32, [i * 7 % 33 - 1 for i in range(64)], 1024, 528, 16, True, "f16", 1.0, 0.0),
    ("bf16", [1] * 70 + [0] * 63 + [3, 2], 2, 3, 5, [i % 6 for i in range(135)], 264, 136, 24, True, "f32", 0.5, 2.0),
    ("bf16", [5, 0, 64, 65, 1, 0], 3, 9, 6, None, 136, 200, 16, True, "f32", 0.5, 2.0),
    ("f16", [5, 0, 64, 65, 1, 0], 3, 9, 6, None, 136, 200, 16, False, "f16", 0.5, 2.0),
    ("bf16", [17, 31, 0, 129], 0, 5, 2, [1, 1, 0, 1], 99, 33, 5, True, "f32", 1.0, 1.0),
    ("f16", [17, 31, 0, 129], 2, 0, 2, [1, -1, 0, 7], 99, 33, 5, False, "bf16", 1.0, 1.0),
    ("bf16", [300, 0, 511, 260], 0, 0, 3, [2, 0, 1, 2], 520, 264, 64, True, "bf16", 1.0, 0.0),
    ("bf16", [300, 0, 511, 260], 0, 7, 4, None, 520, 264, 72, False, "f32", 1.0, 1.0),
    ("f16", [40, 3, 90], 1, 1, 3, None, 200, 136, 130, True, "f32", 1.0, 0.0),
    ("bf16", [40, 3, 90], 1, 1, 3, None, 200, 136, 200, False, "bf16", 1.0, 0.0),
    ("bf16", [100], 0, 0, 0, [-1], 128, 128, 16, True, "bf16", 1.0, 0.0),  # no adapters at all
    ("f16", [600, 700], 0, 0, 2, None, 256, 1032, 32, True, "f16", 1.0, 0.0),
    ("bf16", [1029, 513], 0, 0, 2, [1, 0], 1032, 1024, 48, True, "f32", 1.0, 0.0),
    ("bf16", [2, 1, 0, 5, 16, 17], 0, 0, 6, None, 2048, 512, 16, True, "bf16", 1.0, 0.0),
    ("f16", [30], 0, 2, 4, [3], 4096, 264, 8, True, "f32", 1.0, 1.0),
    ("bf16", [2, 0, 12], 0, 1, 3, None, 1000, 130, 8, False, "bf16", 1.0, 0.0),
    # few rows, more than 64 of them; long and empty requests; ranks that are no granules; the longest
    # part of K, and one k-tile
    ("bf16", [1] * 100 + [0] * 70 + [30], 3, 20, 7, [i * 5 % 9 - 1 for i in range(171)], 1600, 136, 16, True, "bf16", 1.0, 0.0),
    ("f16", [64, 0, 1, 127, 64], 0, 0, 2, [1, 0, 1, 0, -1], 264, 200, 128, True, "f32", 0.5, 1.0),
    ("bf16", [3, 40, 21], 0, 4, 3, None, 64, 72, 5, True, "f32", 1.0, 1.0),
    ("f16", [2, 9], 1, 0, 2, [1, 0], 8, 17, 1, True, "f16", 1.0, 0.0),
    ("bf16", [33, 90, 17], 0, 0, 3, None, 2104, 1100, 33, True, "bf16", 1.0, 0.0),
    ("f16", [20, 12], 0, 0, 2, None, 4160, 64, 48, True, "f32", 1.0, 0.0),
    # few rows by N-contiguous operands, and by operands of any alignment
    ("bf16", [1] * 40 + [0, 20], 1, 2, 5, [i % 6 - 1 for i in range(42)], 1600, 136, 16, False, "bf16", 1.0, 0.0),
    ("f16", [9, 0, 7], 0, 0, 3, None, 4160, 72, 128, False, "f32", 0.5, 1.0),
    ("bf16", [100, 3, 130], 0, 4, 2, [1, 0, 1], 264, 1096, 40, False, "f32", 1.0, 0.0),
    ("f16", [30, 1], 2, 0, 2, None, 1031, 203, 77, False, "f32", 1.0, 1.0),
    ("bf16", [30, 0, 61], 0, 0, 3, [2, 1, 0], 1030, 205, 33, True, "bf16", 1.0, 0.0),
    ("bf16", [200, 40], 0, 5, 2, None, 67, 131, 120, False, "bf16", 1.0, 0.0),
    ("f16", [3], 0, 0, 1, None, 7, 3, 3, False, "f16", 1.0, 0.0),
    # more than 64 of the few rows
    ("bf16", [1] * 60 + [0] * 70 + [30, 31], 3, 4, 7, [i * 5 % 9 - 1 for i in range(132)], 1600, 136, 16, True, "bf16", 1.0, 0.0),
    ("f16", [50, 0, 1, 77], 0, 0, 2, [1, 0, 1, 0], 264, 200, 128, False, "f32", 0.5, 1.0),
    ("bf16", [60, 7, 41], 2, 3, 3, None, 1031, 203, 77, True, "f32", 1.0, 1.0),
    # past the few rows: copies of X and W in whole granules
    ("bf16", [117, 31, 0, 129], 0, 5, 2, [1, 1, 0, 1], 99, 33, 5, True, "f32", 1.0, 1.0),
    ("f16", [117, 31, 0, 129], 2, 0, 2, [1, -1, 0, 7], 99, 33, 5, False, "bf16", 1.0, 1.0),
    ("bf16", [300, 3, 90], 1, 1, 3, None, 200, 136, 130, False, "f32", 1.0, 0.0),
    # staged tiles: many requests, ranks that are no granules, both layouts
    ("bf16", [1, 3] * 90, 2, 1, 5, [i % 6 - 1 for i in range(180)], 136, 264, 13, True, "bf16", 1.0, 0.0),
    ("f16", [1, 3] * 90, 2, 1, 5, [i % 6 - 1 for i in range(180)], 136, 264, 13, False, "f32", 1.0, 1.0),
    ("bf16", [1, 3] * 90, 0, 0, 5, [i % 6 - 1 for i in range(180)], 135, 263, 40, False, "f32", 1.0, 0.0),
    # 128 x 128 tiles, of few and many requests, copied or not
    ("bf16", [500, 0, 7, 590], 2, 1, 4, None, 72, 4104, 16, True, "bf16", 1.0, 0.0),
    ("f16", [500, 0, 7, 590], 0, 4, 3, [2, 0, -1, 1], 99, 4101, 21, False, "f32", 0.5, 1.0),
    ("bf16", [3] * 340, 0, 0, 5, [i % 6 - 1 for i in range(340)], 136, 4104, 40, False, "bf16", 1.0, 0.0),
    ("f16", [3] * 360, 1, 0, 5, [i % 6 - 1 for i in range(360)], 131, 4104, 40, True, "f16", 1.0, 0.0),
    # many requests of one row
    ("bf16", [1] * 1100, 0, 2, 5, [i % 6 - 1 for i in range(1100)], 72, 4104, 16, True, "f32", 1.0, 0.0),
    # 256 x 256 tiles: requests that end inside a tile, a rank of more than one k-tile, both layouts
    ("bf16", [700, 0, 1400, 30], 0, 3, 3, [2, 0, 1, -1], 72, 4104, 16, True, "bf16", 1.0, 0.0),
    ("f16", [700, 0, 1400, 30], 5, 0, 3, [2, 0, -1, 1], 136, 4104, 72, False, "f32", 0.5, 1.0),
    ("bf16", [100, 1, 1900, 255], 0, 0, 2, [0, 1, 1, 0], 200, 4099, 136, True, "f32", 1.0, 0.0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}-q{len(c[1])}-{c[6]}x{c[7]}r{c[8]}-{'linear' if c[9] else 'row'}-{c[10]}")
def test_adapters(dmp, case):
    dt, rows, head, tail, adapters, ids, K, N, r, linear, out, alpha, beta = case
    log(f"[adapters] {case}")
    T = head + sum(rows) + tail
    off = [head] + [int(v) for v in head + np.cumsum(rows)]
    X, W, A, B = operands(1, T, K, N, r, adapters, DT[dt], linear)
    scale = torch.exp2(torch.arange(adapters) % 4 - 2.0)
    C = normal(9, T, N, dtype=DT[out]) if beta else None
    want, tol, h, htol, owned = reference(X, W, A, B, off, ids, scale, alpha, beta, C, DT[out])
    g = [to_gpu(v) for v in (X, W, A, B)]
    o = torch.tensor(off).cuda()
    i = torch.tensor(ids, dtype=torch.int32).cuda() if ids is not None else None
    D = torch.full((T, N), 7.0, dtype=DT[out], device="cuda")
    hidden = torch.full((T, r), 5.0, dtype=DT[dt], device="cuda")
    kw = dict(alpha=alpha, beta=beta)
    c = C.cuda() if beta else None
    res = dmp.gemm_adapters(*g, o, i, scale.cuda(), c, out=D, hidden=hidden, **kw)
    assert res is D
    torch.cuda.synchronize()
    assert (D[~owned.cuda()] == 7).all() and (hidden[~owned.cuda()] == 5).all()
    close(D[owned.cuda()], want[owned], tol[owned], "D")
    close(hidden[owned.cuda()], h[owned], htol[owned], "hidden")
    # 32-bit offsets, no hidden rows for the caller, a new output; the same bits
    D2 = dmp.gemm_adapters(*g, o.int(), i, scale.cuda(), c, out_dtype=DT[out], **kw)
    assert torch.equal(D2[owned.cuda()], D[owned.cuda()])
    # no scale: 1 (a power of two is exact)
    one = dmp.gemm_adapters(*g, o, i, None, c, out_dtype=DT[out], **kw)
    ones = dmp.gemm_adapters(*g, o, i, torch.ones(adapters, device="cuda"), c, out_dtype=DT[out], **kw)
    assert torch.equal(one[owned.cuda()], ones[owned.cuda()])


def test_nothing_to_do(dmp):
    X, W, A, B = (to_gpu(v) for v in operands(1, 6, 16, 24, 8, 2, torch.bfloat16, True))
    off = torch.tensor([2, 2, 2], device="cuda")
    D = torch.full((6, 24), 7.0, device="cuda")
    assert (dmp.gemm_adapters(X, W, A, B, off, out=D) == 7).all()
    off = torch.zeros(1, dtype=torch.int64, device="cuda")
    ids = torch.zeros(0, dtype=torch.int32, device="cuda")
    assert (dmp.gemm_adapters(X, W, A, B, off, ids, out=D) == 7).all()
    X, W, A, B = (to_gpu(v) for v in operands(1, 0, 16, 24, 8, 2, torch.bfloat16, True))
    assert dmp.gemm_adapters(X, W, A, B, torch.zeros(3, dtype=torch.int64, device="cuda")).shape == (0, 24)
    # K == 0: beta * C, hidden rows of zeros
    for linear in (False, True):
        X, W, A, B = (v.cuda() for v in operands(1, 6, 0, 24, 8, 1, torch.bfloat16, linear))
        off = torch.tensor([1, 5], device="cuda")
        C = normal(3, 6, 24).cuda()
        h = torch.full((6, 8), 5.0, dtype=torch.bfloat16, device="cuda")
        D.fill_(7.0)
        dmp.gemm_adapters(X, W, A, B, off, C=C, out=D, beta=2.0, hidden=h)
        assert torch.equal(D[1:5], 2 * C[1:5]) and (D[0] == 7).all() and (D[5] == 7).all()
        assert not h[1:5].any() and (h[0] == 5).all() and (h[5] == 5).all()


def test_offsets_that_are_wrong_stay_inside(dmp):
    """Numbers beyond the rows count as the nearest end; rows are those of the ends."""
    X, W, A, B = (to_gpu(v) for v in operands(1, 200, 64, 128, 8, 3, torch.bfloat16, True))
    want = dmp.gemm_adapters(X, W, A, B, torch.tensor([0, 50, 120, 200], device="cuda"))
    for off in ([-5, 50, 120, 1 << 40], [-(1 << 40), 50, 120, 201]):
        assert torch.equal(dmp.gemm_adapters(X, W, A, B, torch.tensor(off, device="cuda")), want)


@pytest.mark.parametrize("T,K,N", [(90, 136, 264), (150, 136, 264), (150, 133, 264), (1100, 136, 4104), (2200, 136, 4104)])
def test_not_a_number_stays_with_its_rows(dmp, T, K, N):
    """A NaN in one adapter, or in one request's row, reaches no other request (each kernel)."""
    for linear in (True, False):
        X, W, A, B = (to_gpu(v) for v in operands(1, T, K, N, 16, 3, torch.bfloat16, linear))
        off = torch.tensor([0, 10, 70, T], device="cuda")
        want = dmp.gemm_adapters(X, W, A, B, off)
        A2, B2 = A.clone(), B.clone()
        A2[1] = float("nan")
        B2[1] = float("inf")
        got = dmp.gemm_adapters(X, W, A2, B2, off)
        assert torch.equal(got[:10], want[:10]) and torch.equal(got[70:], want[70:]) and got[10:70].isnan().all()
        X2 = X.clone()
        X2[20] = float("nan")
        got = dmp.gemm_adapters(X2, W, A, B, off)
        assert torch.equal(got[:20], want[:20]) and torch.equal(got[21:], want[21:]) and got[20].isnan().all()


def test_large_hidden_values(dmp):
    """h beyond fp16: an infinity, in 16-bit and in 32-bit results, and no NaN from its rest."""
    X = torch.full((3, 64), 8.0, dtype=torch.float16, device="cuda")
    W = torch.zeros(128, 64, dtype=torch.float16, device="cuda").t()
    A = torch.full((1, 8, 64), 200.0, dtype=torch.float16, device="cuda").transpose(1, 2)
    B = torch.full((1, 128, 8), 1.0, dtype=torch.float16, device="cuda").transpose(1, 2)
    off = torch.tensor([0, 3], device="cuda")
    for out in (torch.float32, torch.float16):
        assert (dmp.gemm_adapters(X, W, A, B, off, out_dtype=out) == float("inf")).all()


def test_strided_operands(dmp):
    """Rows of every operand and of the results further apart than they are long; D over C."""
    off = torch.tensor([0, 30, 100], device="cuda")
    for linear in (True, False):
        X, W, A, B = operands(4, 100, 72, 136, 16, 2, torch.bfloat16, linear)
        want = dmp.gemm_adapters(*(to_gpu(v) for v in (X, W, A, B)), off, out_dtype=torch.bfloat16)

        def wide(x):
            t = x.transpose(-1, -2) if x.stride(-1) != 1 else x
            big = torch.full((*t.shape[:-1], t.shape[-1] + 24), float("nan"), dtype=t.dtype, device="cuda")
            big[..., 8:8 + t.shape[-1]] = t.cuda()
            v = big[..., 8:8 + t.shape[-1]]
            return v.transpose(-1, -2) if x.stride(-1) != 1 else v

        D = torch.full((100, 200), 7.0, dtype=torch.bfloat16, device="cuda")
        dmp.gemm_adapters(*(wide(v) for v in (X, W, A, B)), off, out=D[:, 40:176])
        assert torch.equal(D[:, 40:176], want) and (D[:, :40] == 7).all() and (D[:, 176:] == 7).all()
        C = normal(8, 100, 136).cuda()
        both = dmp.gemm_adapters(*(to_gpu(v) for v in (X, W, A, B)), off, C=C)
        got = dmp.gemm_adapters(*(to_gpu(v) for v in (X, W, A, B)), off, C=C, out=C)
        assert got is C and torch.equal(C, both)


@pytest.mark.parametrize("T", [100, 300])
def test_operands_that_begin_anywhere(dmp, T):
    """Views that start at odd elements, rows of odd lengths apart, NaN around them, one operand and all of
    them: the bits of the same numbers side by side."""
    off = torch.tensor([0, 30, 100, T], device="cuda")
    for linear in (True, False):
        ops = [to_gpu(v) for v in operands(4, T, 69, 131, 13, 3, torch.bfloat16, linear)]

        def odd(x):
            t = x.transpose(-1, -2) if x.stride(-1) != 1 else x
            n = t.shape[-1] + 5
            flat = torch.full((t[..., 0].numel() * n + 3,), float("nan"), dtype=t.dtype, device="cuda")
            v = flat[3:].view(*t.shape[:-1], n)[..., :t.shape[-1]]
            v.copy_(t)
            return v.transpose(-1, -2) if x.stride(-1) != 1 else v

        want = dmp.gemm_adapters(*ops, off, out_dtype=torch.bfloat16)
        for which in ((0,), (1,), (2,), (3,), (0, 1, 2, 3)):
            got = dmp.gemm_adapters(*(odd(v) if i in which else v for i, v in enumerate(ops)), off, out_dtype=torch.bfloat16)
            assert torch.equal(got, want), which


@pytest.mark.parametrize("linear", [True, False])
def test_gradients(dmp, linear):
    """The documented composition against the formulas in 64 bits; padding rows in front and behind."""
    dt, T, K, N, r, a = torch.bfloat16, 400, 136, 200, 24, 3
    off = [3, 90, 90, 390]
    X, W, A, B = operands(11, T, K, N, r, a, dt, linear)
    scale = torch.tensor([0.5, 1.0, 2.0])
    dY = normal(20, T, N, dtype=dt)
    g = [to_gpu(v) for v in (X, W, A, B)]
    o, sc, dy = torch.tensor(off).cuda(), scale.cuda(), dY.cuda()
    h = torch.empty(T, r, dtype=dt, device="cuda")
    gh = torch.empty_like(h)
    dmp.gemm_adapters(*g, o, scale=sc, hidden=h)
    dX = dmp.gemm_adapters(dy, g[1].t(), g[3].transpose(1, 2), g[2].transpose(1, 2), o, scale=sc, hidden=gh, out_dtype=dt)
    dA, dB = dmp.gemm_grouped_wgrad(g[0], gh, o), dmp.gemm_grouped_wgrad(h, dy, o)
    want, tol, gw, gtol, owned = reference(dY, W.t(), B.transpose(1, 2), A.transpose(1, 2), off, None, scale, 1.0, 0.0, None, dt)
    close(dX[owned.cuda()], want[owned], tol[owned], "dX")
    _, _, hw, htol, _ = reference(X, W, A, B, off, None, scale, 1.0, 0.0, None, dt)
    x, y = X.double(), dY.double()
    for i in range(a):
        s = slice(off[i], off[i + 1])
        n = off[i + 1] - off[i]
        # the hidden rows' errors through the sums, and 4 n u of the sums themselves
        close(dA[i], x[s].t() @ gw[s], x[s].abs().t() @ gtol[s] + 4 * n * U * (x[s].abs().t() @ (gw[s].abs() + gtol[s])) * 1.01 + 1e-30, "dA")
        close(dB[i], hw[s].t() @ y[s], htol[s].t() @ y[s].abs() + 4 * n * U * ((hw[s].abs() + htol[s]).t() @ y[s].abs()) * 1.01 + 1e-30, "dB")


def test_formulas_against_differences():
    """The gradients' formulas themselves, in 64 bits on the CPU, against central differences."""
    X, W, A, B = (v.double() for v in operands(30, 7, 6, 5, 3, 2, torch.float32, False))
    off, scale, dY = [0, 4, 7], [0.5, 2.0], normal(31, 7, 5).double()

    def loss(x, a, b):
        y = x @ W
        for g in range(2):
            s = slice(off[g], off[g + 1])
            y[s] = y[s] + scale[g] * (x[s] @ a[g]) @ b[g]
        return float((y * dY).sum())

    dX = dY @ W.t()
    dA, dB = torch.zeros_like(A), torch.zeros_like(B)
    for g in range(2):
        s = slice(off[g], off[g + 1])
        dX[s] += scale[g] * (dY[s] @ B[g].t()) @ A[g].t()
        dA[g] = scale[g] * X[s].t() @ (dY[s] @ B[g].t())
        dB[g] = scale[g] * (X[s] @ A[g]).t() @ dY[s]
    eps = 1e-6
    for which, grad in ((0, dX), (1, dA), (2, dB)):
        args = [X, A, B]
        flat = grad.flatten()
        for i in range(0, flat.numel(), 5):
            v = []
            for sign in (1, -1):
                moved = args[which].clone()
                moved.view(-1)[i] += sign * eps
                v.append(loss(*[moved if j == which else args[j] for j in range(3)]))
            assert abs((v[0] - v[1]) / (2 * eps) - flat[i]) < 1e-7


@pytest.mark.parametrize("T", [120, 300])
def test_streams_and_captured_graphs(dmp, T):
    """Each call has scratch of its own, on two streams and in two graphs replayed in turn; a graph
    follows the offsets and adapters that are there at replay."""
    off = torch.tensor([0, 30, 100, T], device="cuda")
    ids = torch.tensor([1, 0, -1], dtype=torch.int32, device="cuda")
    sets = [[to_gpu(v) for v in operands(40 + i, T, 264, 136, 16, 2, torch.bfloat16, i == 0)] for i in range(2)]
    want = [dmp.gemm_adapters(*s, off, ids) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(8):
        with torch.cuda.stream(streams[i % 2]):
            got.append(dmp.gemm_adapters(*sets[i % 2], off, ids))
    torch.cuda.synchronize()
    assert all(torch.equal(v, want[i % 2]) for i, v in enumerate(got))
    graphs, outs = [], []
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(dmp.gemm_adapters(*sets[i], off, ids))
        graphs.append(graph)
    for i, (o, a) in enumerate([([0, 30, 100, T], [1, 0, -1]), ([0, 0, T, T], [0, 1, 1]), ([0, 1, 2, T], [1, 1, 0]),
                                ([0, T - 1, T - 1, T], [-1, 1, 0])]):
        off.copy_(torch.tensor(o))
        ids.copy_(torch.tensor(a, dtype=torch.int32))
        for j in range(2):
            graphs[j].replay()
            torch.cuda.synchronize()
            assert torch.equal(outs[j], dmp.gemm_adapters(*sets[j], off, ids))
