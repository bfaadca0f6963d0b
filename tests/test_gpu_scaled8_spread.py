"""8-bit products of values that span many powers of two within 8 consecutive k, which is
where the 8-bit matrix instruction drops what lies 13 bits below the largest product.

Tolerance per element, from the header: 4 (K + 128) 2^-24 S, with 16-bit results of more
than a few rows 2^-9 S more (S: the sum of the scaled products' magnitudes), three fp32 roundings
of the output stage and half a step of the output type, at least half its least subnormal."""
import pytest

from gpu_util import log
from test_gpu_scaled8 import E4, E5, dmp  # noqa: F401

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

OUT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
TINY = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
FORMATS = [(E4, E4), (E5, E5), (E5, E4), (E4, E5)]
# the 16-bit results of the first run in 128 x 128 tiles, of the second in 256 x 256 ones, of
# the third in the kernel for few rows, which widens the values whatever the result
SIZES = [(200, 384, 264), (4100, 272, 4100), (12, 384, 264)]


def powers(seed, rows, K, lo, hi):
    """Signed powers of two, exponents evenly from lo .. hi."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    e = torch.randint(lo, hi + 1, (rows, K), generator=g, device="cuda").float()
    sign = torch.randint(0, 2, (rows, K), generator=g, device="cuda").float() * 2 - 1
    return torch.exp2(e) * sign


def cancelling(T, N, K, low, fmt_a, fmt_b):
    """In each 8 consecutive k two products of 2^16 that cancel, in places that move on from
    one 8 to the next, and six of 2^(16 - low)."""
    a, b = powers(1, T, K, 0, 0), powers(2, N, K, 0, 0)
    half = low // 2
    a *= 2.0 ** (8 - half)
    b *= 2.0 ** (8 - (low - half))
    k = torch.arange(K, device="cuda")
    one, other = k % 8 == (k // 8) % 8, k % 8 == (k // 8 + 3) % 8
    a[:, one | other], b[:, one], b[:, other] = 256.0, 256.0, -256.0
    return a, b


def run(dmp, a, b, K, out, few):  # noqa: F811
    """Compares with 64 bits; returns the error's norm over S's."""
    T, N = a.shape[0], b.shape[0]
    scale = 2.0 ** -10  # (fp16 results stay finite)
    A = dmp.Scaled8(a, torch.full((T, -(-K // 128)), scale, device="cuda"), K=K)
    B = dmp.Scaled8(b, torch.full((-(-N // 128), -(-K // 128)), scale, device="cuda"), block=128, K=K)
    D = dmp.gemm_scaled8(A, B, out_dtype=out).double()
    a, b = a[:, :K].double() * scale, b[:, :K].double() * scale
    acc, S = a @ b.t().contiguous(), a.abs() @ b.abs().t().contiguous()
    u = 2.0 ** -24
    tol = 1.01 * (4 * (K + 128) * u * S + 3 * u * acc.abs() + torch.finfo(out).eps / 2 * acc.abs()) + TINY[out]
    if out != torch.float32 and not few:
        tol += 2.0 ** -9 * S
    assert torch.isfinite(D).all()
    bad = (D - acc).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} over the bound, worst {float(((D - acc).abs() / tol).max()):.3g}"
    return float((D - acc).norm() / S.norm())


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("fa,fb", FORMATS, ids=["e4e4", "e5e5", "e5e4", "e4e5"])
@pytest.mark.parametrize("T,K,N", SIZES)
def test_cancelling_products_beside_small_ones(dmp, T, K, N, fa, fb, out):  # noqa: F811
    for low in (8, 11, 12, 13, 14, 15, 18):
        a, b = cancelling(T, N, K, low, fa, fb)
        r = run(dmp, a.to(fa), b.to(fb), K, OUT[out], T <= 16)
        log(f"[scaled8] cancelling {T}x{K}x{N} {fa} {fb} {out} low 2^-{low}: {r:.2e} of S")


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("fa,fb", FORMATS, ids=["e4e4", "e5e5", "e5e4", "e4e5"])
@pytest.mark.parametrize("T,K,N", SIZES)
def test_products_over_many_powers_of_two(dmp, T, K, N, fa, fb, out):  # noqa: F811
    r = run(dmp, powers(3, T, K, -8 if fa == E4 else -12, 8).to(fa), powers(4, N, K, -8 if fb == E4 else -12, 8).to(fb), K,
            OUT[out], T <= 16)
    log(f"[scaled8] powers of two {T}x{K}x{N} {fa} {fb} {out}: {r:.2e} of S")
