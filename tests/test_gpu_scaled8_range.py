"""8-bit products whose factors are far from one: sA * sB below the normal numbers or
above the largest float, where the scaled sums are ordinary numbers.

Tolerance per element: the header's 4 (K + 128) 2^-24 S, with 16-bit results 2^-9 S more, three fp32
roundings of the output stage and half a step of the output type (S: the sum of the scaled
products' magnitudes).  No scaled sum here leaves fp32's normal numbers."""
import pytest

from gpu_util import log
from test_gpu_scaled8 import E4, E5, TOP, dmp  # noqa: F401

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

# rows, K, N: few rows with 16, 32 and 64 columns to a workgroup; 128 x 128 tiles; the largest tiles
SIZES = [(3, 384, 200), (20, 400, 8200), (16, 272, 16400), (200, 384, 264), (4100, 272, 4100)]
OUT = {"f32": torch.float32, "bf16": torch.bfloat16}


def normal(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda")


def values(q, scale, block, K):
    s = scale.double().repeat_interleave(128, -1)[:, :K]
    return q[:, :K].double() * (s.repeat_interleave(block, 0)[:q.shape[0]] if block > 1 else s)


def within_bound(D, a, b, K, out, keep=slice(None)):
    acc, S = a @ b.t().contiguous(), a.abs() @ b.abs().t().contiguous()
    u = 2.0 ** -24
    tol = 1.01 * (4 * (K + 128) * u * S + 3 * u * acc.abs() + torch.finfo(out).eps / 2 * acc.abs())
    if out != torch.float32:
        tol += 2.0 ** -9 * S
    got, ref, tol = D.double()[keep], acc[keep], tol[keep]
    assert torch.isfinite(got).all()
    bad = (got - ref).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} over the bound, worst {float(((got - ref).abs() / tol).max()):.3g}"


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("fa,fb", [(E4, E4), (E5, E5), (E5, E4)], ids=["e4e4", "e5e5", "e5e4"])
@pytest.mark.parametrize("T,K,N", SIZES)
def test_products_of_factors_below_the_normal_numbers(dmp, T, K, N, fa, fb, out):  # noqa: F811
    """Every third row meets factors of 2^-140 and less (some of them 0 in fp32) in every
    second block of 128 columns, the other rows ordinary ones."""
    log(f"[scaled8] small factors {T}x{K}x{N} {fa} {fb} {out}")
    kp, kb, nb = -(-K // 16) * 16, -(-K // 128), -(-N // 128)
    a = (normal(1, T, kp) * (TOP[fa] / 4)).clamp(-TOP[fa], TOP[fa])
    b = (normal(2, N, kp) * (TOP[fb] / 4)).clamp(-TOP[fb], TOP[fb])
    a[:, K:], b[:, K:] = 0, 0
    a, b = a.to(fa), b.to(fb)
    # e4m3 values reach 2^8.8, e5m2 values 2^15.8: factors as small as the sums allow
    low = -70 - (4 if fa == E5 else 0) - (4 if fb == E5 else 0)
    sa, sb = torch.exp2(normal(3, T, kb)), torch.exp2(normal(4, nb, kb))
    sa[::3] *= 2.0 ** low
    sb[::2] *= 2.0 ** -70
    A, B = dmp.Scaled8(a, sa, K=K), dmp.Scaled8(b, sb, block=128, K=K)
    D = dmp.gemm_scaled8(A, B, out_dtype=OUT[out])
    within_bound(D, values(a, sa, 1, K), values(b, sb, 128, K), K, OUT[out])
    # the rows beside: bit for bit what they are among ordinary rows
    sa[::3] = 1.0
    E = dmp.gemm_scaled8(A, B, out_dtype=OUT[out])
    keep = torch.arange(T) % 3 != 0
    assert torch.equal(D[keep], E[keep])


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("T,K,N", SIZES)
def test_products_of_factors_above_the_largest_float(dmp, T, K, N, out):  # noqa: F811
    """Factors of 2^130 and more by 8-bit values of 2^-16: sums of about 2^100; and rows of
    zeros, whose results are zero."""
    log(f"[scaled8] large factors {T}x{K}x{N} {out}")
    kp, kb, nb = -(-K // 16) * 16, -(-K // 128), -(-N // 128)
    sign = [torch.sign(normal(s, n, kp)) * 2.0 ** -16 for s, n in ((5, T), (6, N))]
    for x in sign:
        x[:, K:] = 0
    sign[0][1::4] = 0
    a, b = sign[0].to(E5), sign[1].to(E5)
    sa, sb = torch.exp2(normal(7, T, kb)), torch.exp2(normal(8, nb, kb))
    sa[::2] *= 2.0 ** 66
    sa[1::4] *= 2.0 ** 100
    sb *= 2.0 ** 66
    A, B = dmp.Scaled8(a, sa, K=K), dmp.Scaled8(b, sb, block=128, K=K)
    D = dmp.gemm_scaled8(A, B, out_dtype=OUT[out])
    assert not D[1::4].any()
    within_bound(D, values(a, sa, 1, K), values(b, sb, 128, K), K, OUT[out])


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("counts", [[2, 0, 5], [200, 0, 130]], ids=["few", "tiles"])
def test_grouped_and_subnormal_factors(dmp, counts, out):  # noqa: F811
    """Subnormal factors by large ones (their product is ordinary), a zero factor, and a
    group whose factors' products underflow."""
    K, N, G, T = 256, 136, len(counts), sum(counts)
    a, b = normal(9, T, K).clamp(-8, 8).to(E4), normal(10, G, N, K).clamp(-8, 8).to(E4)
    sa, sb = torch.full((T, 2), 2.0 ** -135, device="cuda"), torch.full((G, 2, 2), 2.0 ** 120, device="cuda")
    sa[0, 0], sb[2, 1, 1] = 0.0, 0.0
    sb[2, 0] = 2.0 ** 20  # 2^-115 with the factor of the rows: normal, sums of 2^-110
    sb[2, 1, 0] = 2.0 ** 8  # 2^-127: subnormal
    off = torch.tensor([0, counts[0], counts[0] + counts[1], T], device="cuda")
    A, B = dmp.Scaled8(a, sa), dmp.Scaled8(b, sb, block=128)
    D = dmp.gemm_scaled8(A, B, off, out_dtype=OUT[out])
    for g, part in ((0, slice(0, counts[0])), (2, slice(counts[0], T))):
        va, vb = values(a[part], sa[part], 1, K), values(b[g], sb[g], 128, K)
        S = va.abs() @ vb.abs().t().contiguous()
        assert float(S.min()) > 2.0 ** -125
        within_bound(D[part], va, vb, K, OUT[out])
