"""The experts' router (route, route_grad) on the GPU against a plain 64-bit computation.

Tolerances, from the arithmetic alone (u = 2^-24, D the spread of a token's available
logits, V = E / 64 logits to a lane).  exp(x - m): x - m is rounded (an error of D u in
the exponent at most) and expf is good to 2 u, so that exp(x - m) is good to (D + 2) u,
relatively, their sum over a lane and six steps of the wave to (D + 2 + V + 6) u, and a
weight, with two roundings more, to (2 D + V + 14) u.  lse adds logf (2 u of its result) and
a rounding.  A loss is a sum over tokens: 16 waves of a workgroup in turn, the workgroups
over up to 16 parts: (tokens / 16 + 48) u more than its terms at most.  A gradient is a sum of four
products of such factors: 4 times a weight's tolerance of the sum of their magnitudes
(and 40 u for the wave's sums and the roundings), and half a step of its type."""
import math

import pytest

import route_reference as ref
from gpu_util import log

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
U = 2.0 ** -24


@pytest.fixture(scope="module")
def dmp():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import dense_mixed_precision_02_amd as dmp
    return dmp


def make_logits(seed, T, E, dtype, spread=1.5, absent=0.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, E, generator=g) * spread + torch.randn(E, generator=g) * 0.5
    if absent:
        x = x.masked_fill(torch.rand(T, E, generator=g) < absent, -math.inf)
    return x.to(DT[dtype])


def spread_of(x):
    x = x.double()
    x = x[torch.isfinite(x)]
    return float(x.max() - x.min()) if x.numel() else 0.0


def check_all(dmp, x, k, mask, normalize, seed=5, balance=0.01, z=0.001, device_x=None):
    T, E = x.shape
    xd = x.cuda() if device_x is None else device_x
    md = mask.cuda() if mask is not None else None
    r = dmp.route(xd, k, mask=md, normalize=normalize)
    experts, order, place, counts, offsets = ref.choose(x, k, mask)
    assert torch.equal(r.experts.cpu(), experts)
    assert torch.equal(r.counts.cpu(), counts)
    assert torch.equal(r.offsets.cpu(), offsets)
    assert torch.equal(r.order.cpu(), order)
    assert torch.equal(r.place.cpu(), place)
    p, lse, w = ref.softmax_parts(x, experts, normalize, mask)
    V, D = -(-E // 64), spread_of(x)
    rel = (2 * D + V + 14) * U
    got = r.weights.cpu().double()
    assert torch.isfinite(got).all()
    # results below the normal floats: expf and the products may flush or round there
    assert ((got - w).abs() <= rel * w + 2.0 ** -125).all()
    live = lse != math.inf
    got = r.lse.cpu().double()
    assert torch.equal(got == math.inf, ~live)
    tol_lse = (D + V + 10) * U + 3 * U * lse[live].abs()
    assert ((got[live] - lse[live]).abs() <= tol_lse).all()
    b, zz = ref.losses(p, lse, counts)
    more = (T / 16 + 48) * U
    loss = r.loss.cpu().double()
    assert abs(loss[0] - b) <= (rel + more) * b
    worst = float((2 * lse[live].abs() * tol_lse).max()) if live.any() else 0.0
    if zz > torch.finfo(torch.float32).max:  # lse^2 of the largest logits: beyond what the result can hold
        assert loss[1] == math.inf
    else:
        assert abs(loss[1] - zz) <= worst + more * zz
    g = torch.Generator().manual_seed(seed)
    dw = torch.randn(T, k, generator=g)
    for d_weights in (dw, None):
        d, size = ref.gradient(x, experts, counts, normalize, d_weights, balance, z, mask)
        got = dmp.route_grad(r, d_weights.cuda() if d_weights is not None else None, balance, z)
        assert got.dtype == x.dtype and got.shape == x.shape
        got = got.cpu().double()
        low = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -125}[x.dtype]
        tol = (4 * rel + 40 * U) * size + torch.finfo(x.dtype).eps / 2 * d.abs() * 1.01 + low
        bad = (got - d).abs() > tol
        assert torch.isfinite(got).all() and not bad.any(), f"{int(bad.sum())} gradients off"
    return r


# T, E, k, dtype, share of masked tokens, share of absent experts, spread, normalize
CASES = [
    (1, 1, 1, "f32", 0, 0, 1.5, False),
    (1, 4, 2, "bf16", 0, 0, 1.5, True),
    (3, 5, 5, "f16", 0, 0.3, 1.5, False),
    (16, 32, 4, "f32", 0, 0, 1.5, True),
    (64, 64, 8, "bf16", 0.3, 0, 1.5, True),
    (65, 63, 6, "f16", 0.3, 0.5, 1.5, False),
    (100, 65, 3, "bf16", 0, 0.9, 1.5, True),
    (257, 64, 64, "f32", 0, 0, 1.5, True),
    (500, 128, 8, "bf16", 0.1, 0, 0.2, False),
    (700, 129, 7, "f32", 0.9, 0.5, 4.0, True),
    (300, 256, 8, "f16", 0, 0, 1.5, True),
    (333, 257, 9, "bf16", 0.1, 0.2, 1.5, False),
    (150, 513, 33, "f32", 0, 0.1, 1.5, True),
    (130, 1023, 5, "bf16", 0.2, 0, 1.5, False),
    (70, 1024, 64, "f32", 0.2, 0.99, 8.0, True),
    (5003, 8, 2, "bf16", 0.1, 0, 1.5, True),
    (4100, 160, 6, "f32", 0.05, 0.5, 1.0, True),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}x{c[1]}k{c[2]}-{c[3]}")
def test_route(dmp, case):
    T, E, k, dtype, masked, absent, spread, normalize = case
    log(f"[route] {case}")
    x = make_logits(T + E, T, E, dtype, spread, absent)
    g = torch.Generator().manual_seed(T)
    mask = torch.rand(T, generator=g) >= masked if masked else None
    check_all(dmp, x, k, mask, normalize)


def test_ties_signs_and_ends(dmp):
    """Equal logits (the lower expert first), zeros of both signs, the types' largest and lowest
    values, subnormals."""
    inf = math.inf
    for dtype in ("f32", "bf16", "f16"):
        fi = torch.finfo(DT[dtype])
        rows = [[1.0] * 70, [0.0, -0.0] * 35, [-0.0, 0.0] * 35, [float(i % 3) for i in range(70)],
                [fi.min] * 70, [fi.min] * 69 + [-inf], [-inf] * 69 + [fi.min], [-inf] * 70,
                [-inf] * 35 + [fi.tiny] * 35, [fi.smallest_normal / 2] * 10 + [0.0] * 60]
        x = torch.tensor(rows).to(DT[dtype])
        for normalize in (False, True):
            check_all(dmp, x, 5, None, normalize)
    # the largest value next to the lowest: their difference is an infinity in 32 bits, and exp of it 0
    x = torch.tensor([[3e38, -3e38, 3e38, 0.0]])
    r = dmp.route(x.cuda(), 3, normalize=True)
    assert r.experts.tolist() == [[0, 2, 3]] and r.weights.tolist() == [[0.5, 0.5, 0.0]]


def test_masked_logits_are_not_looked_at(dmp):
    """A masked token may hold anything; its gradient is zero."""
    x = make_logits(3, 40, 20, "f32")
    mask = torch.ones(40, dtype=torch.bool)
    mask[7] = mask[39] = False
    bad = x.clone()
    bad[7], bad[39] = math.nan, math.inf
    a, b = (dmp.route(v.cuda(), 3, mask=mask.cuda()) for v in (x, bad))
    for name in ("experts", "weights", "counts", "order", "place", "loss", "lse"):
        assert torch.equal(getattr(a, name), getattr(b, name)), name
    dw = torch.ones(40, 3, device="cuda")
    assert torch.equal(dmp.route_grad(a, dw, 0.1, 0.1), dmp.route_grad(b, dw, 0.1, 0.1))
    assert not dmp.route_grad(b, dw, 0.1, 0.1)[7].any()


def test_numbers_that_are_none_show(dmp):
    """A NaN or +inf: the token's weights and the losses are NaN, tables stay whole."""
    for value in (math.nan, math.inf):
        x = make_logits(4, 33, 12, "bf16")
        x[5, 3] = value
        r = dmp.route(x.cuda(), 2)
        assert r.weights[5].isnan().all() and r.lse[5].isnan() and r.loss.isnan().all()
        assert not r.weights[:5].isnan().any() and not r.weights[6:].isnan().any()
        assert int(r.counts.sum()) == 66 and sorted(r.order.tolist()) == list(range(66))
        assert (3 in r.experts[5].tolist()) == (value == math.inf)
        assert dmp.route_grad(r, torch.ones(33, 2, device="cuda"))[5].isnan().all()
    x = torch.full((2, 6), -math.inf)
    x[0, 2] = math.nan  # nothing but a NaN
    r = dmp.route(x.cuda(), 2)
    assert r.experts.tolist() == [[-1, -1]] * 2 and r.loss.isnan().all()


def test_no_tokens(dmp):
    for T, mask in ((0, None), (0, torch.zeros(0, dtype=torch.bool)), (5, torch.zeros(5, dtype=torch.bool)),
                    (200, torch.zeros(200, dtype=torch.bool))):
        x = make_logits(1, T, 9, "f32")
        check_all(dmp, x, 2, mask, True)
        r = dmp.route(x.cuda(), 2, mask=mask.cuda() if mask is not None else None)
        assert r.counts.tolist() == [0] * 9 and r.offsets.tolist() == [0] * 10 and r.loss.tolist() == [0.0, 0.0]


def test_strided_rows_and_outputs(dmp):
    """Rows further apart than E; a gradient into rows that are, and over the logits."""
    wide = make_logits(8, 90, 50, "bf16").cuda()
    x = wide[:, 3:33]
    r = check_all(dmp, x.cpu(), 4, None, True, device_x=x)
    dw = torch.randn(90, 4, device="cuda")
    d = dmp.route_grad(r, dw, 0.1, 0.2)
    out = torch.full((90, 50), 7.0, dtype=torch.bfloat16, device="cuda")
    assert dmp.route_grad(r, dw, 0.1, 0.2, out=out[:, 10:40]) is not None
    assert torch.equal(out[:, 10:40], d) and (out[:, :10] == 7).all() and (out[:, 40:] == 7).all()
    dmp.route_grad(r, dw, 0.1, 0.2, out=x)
    assert torch.equal(x, d) and torch.equal(wide[:, 33:].cpu(), make_logits(8, 90, 50, "bf16")[:, 33:])


def test_repeats_and_streams(dmp):
    """The same bits every time, and on two streams at once."""
    x = make_logits(9, 3000, 64, "f32").cuda()
    dw = torch.randn(3000, 4, device="cuda")
    a = dmp.route(x, 4)
    da = dmp.route_grad(a, dw, 0.1, 0.1)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):
            r = dmp.route(x, 4)
            got.append((r, dmp.route_grad(r, dw, 0.1, 0.1)))
    torch.cuda.synchronize()
    for r, d in got:
        assert torch.equal(d, da)
        for name in ("experts", "weights", "counts", "offsets", "order", "place", "loss", "lse"):
            assert torch.equal(getattr(r, name), getattr(a, name)), name


def test_captured_graph_follows_its_inputs(dmp):
    x = make_logits(10, 2000, 32, "bf16").cuda()
    mask = torch.ones(2000, dtype=torch.bool, device="cuda")
    dw = torch.randn(2000, 2, device="cuda")
    dmp.route_grad(dmp.route(x, 2, mask=mask), dw, 0.1, 0.1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = dmp.route(x, 2, mask=mask)
        d = dmp.route_grad(r, dw, 0.1, 0.1)
    for i in range(4):
        x.copy_(make_logits(20 + i, 2000, 32, "bf16"))
        mask.copy_(torch.rand(2000) > 0.1 * i)
        graph.replay()
        torch.cuda.synchronize()
        e = dmp.route(x, 2, mask=mask)
        assert torch.equal(d, dmp.route_grad(e, dw, 0.1, 0.1))
        for name in ("experts", "weights", "counts", "offsets", "order", "place", "loss", "lse"):
            assert torch.equal(getattr(r, name), getattr(e, name)), name


def test_layer(dmp):
    """The router in front of the experts' products, as a layer uses them: gather, product, weighted
    sum, and the weight gradients; padding tokens and tokens with fewer experts than k."""
    T, E, k, K, N = 300, 12, 3, 64, 72
    g = torch.Generator().manual_seed(1)
    x = make_logits(11, T, E, "f32", absent=0.7)
    mask = torch.rand(T, generator=g) > 0.2
    X = torch.randn(T, K, generator=g).bfloat16()
    W = (torch.randn(E, K, N, generator=g) / 8).bfloat16()
    r = dmp.route(x.cuda(), k, mask=mask.cuda(), normalize=True)
    rows = X.cuda()[r.order // k]
    Y = dmp.gemm_grouped(rows, W.cuda(), r.offsets, out=torch.zeros(T * k, N, device="cuda"))
    D = (Y[r.place.long()].view(T, k, N) * r.weights[..., None]).sum(1)
    experts, *_ = ref.choose(x, k, mask)
    _, _, w = ref.softmax_parts(x, experts, True, mask)
    Xd, Wd = X.double(), W.double()
    want, size = torch.zeros(T, N, dtype=torch.float64), torch.zeros(T, N, dtype=torch.float64)
    grad = torch.zeros(E, K, N, dtype=torch.float64)
    gsize = torch.zeros(E, K, N, dtype=torch.float64)
    dY = torch.randn(T * k, N, generator=g).bfloat16()
    place = r.place.cpu()
    for t in range(T):
        for j in range(k):
            e = int(experts[t, j])
            if e >= 0:
                want[t] += w[t, j] * (Xd[t] @ Wd[e])
                size[t] += w[t, j] * (Xd[t].abs() @ Wd[e].abs())
                o = dY[place[t * k + j]].double()
                grad[e] += torch.outer(Xd[t], o)
                gsize[e] += torch.outer(Xd[t].abs(), o.abs())
    # products: 4 K u; the weights and the sum of k of them: (2 D + 20) u
    assert ((D.cpu().double() - want).abs() <= (4 * K + 2 * spread_of(x) + 20) * U * size).all()
    dW = dmp.gemm_grouped_wgrad(rows, dY.cuda(), r.offsets)
    assert ((dW.cpu().double() - grad).abs() <= 4 * T * U * gsize + 1e-30).all()
