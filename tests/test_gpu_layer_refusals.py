"""Refusals of the torch front ends that need tensors on a GPU to get that far: nothing is
launched."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dmp():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import dense_mixed_precision_02_amd as dmp
    return dmp


def test_adapters(dmp):
    def call(**kw):
        t = dict(X=torch.zeros(4, 8), W=torch.zeros(8, 16), A=torch.zeros(2, 8, 4), B=torch.zeros(2, 4, 16))
        a = {k: kw.pop(k) if k in kw else v.half().cuda() for k, v in t.items()}
        off = kw.pop("offsets", torch.tensor([0, 2, 4], device="cuda"))
        return dmp.gemm_adapters(a["X"], a["W"], a["A"], a["B"], off, **kw)

    z = lambda *s, dtype=torch.float16: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    call()
    for bad in (dict(A=z(2, 8, 4, dtype=torch.bfloat16)), dict(B=z(2, 4, 16, dtype=torch.float32)),
                dict(ids=z(2, dtype=torch.int64)), dict(scale=z(2)), dict(hidden=z(4, 4, dtype=torch.float32)),
                dict(offsets=z(3, dtype=torch.float32)), dict(out=z(4, 16, dtype=torch.float64))):
        with pytest.raises(TypeError):
            call(**bad)
    for bad in (dict(A=z(2, 9, 4)), dict(B=z(3, 4, 16)), dict(B=z(2, 5, 16)), dict(W=z(9, 16)), dict(W=z(8, 16, 1)),
                dict(offsets=torch.tensor([0, 4], device="cuda")), dict(offsets=torch.tensor([0, 2, 4])),
                dict(ids=z(3, dtype=torch.int32)), dict(ids=torch.zeros(2, dtype=torch.int32)), dict(ids=z(4, dtype=torch.int32)[::2]),
                dict(scale=z(3, dtype=torch.float32)), dict(hidden=z(4, 5)), dict(hidden=z(4, 4).t()), dict(A=z(2, 8, 0), B=z(2, 0, 16)),
                dict(W=z(16, 8).t()),  # W and B laid out differently
                dict(A=z(4, 8, 4)[::2]), dict(B=z(2, 4, 32)[:, :, ::2]), dict(C=z(4, 16)[:, ::2], out=z(4, 8)),
                dict(A=z(2, 8, 1025), B=z(2, 1025, 16))):
        with pytest.raises(ValueError):
            call(**bad)
    ids = torch.tensor([1], dtype=torch.int32, device="cuda")  # fewer requests than adapters: ids say which
    call(offsets=torch.tensor([0, 4], device="cuda"), ids=ids)


def test_wgrad8_and_quant8(dmp):
    x = dmp.quant8(torch.zeros(6, 20, device="cuda"), pow2=True)
    y = torch.zeros(6, 8, dtype=torch.bfloat16, device="cuda")
    assert dmp.gemm_wgrad8(x, y).shape == (20, 8)
    with pytest.raises(TypeError):
        dmp.gemm_wgrad8(x, y.float())
    for bad in (y[:5], y.cpu(), y.t(), y[None]):
        with pytest.raises(ValueError):
            dmp.gemm_wgrad8(x, bad)
    with pytest.raises(ValueError):  # blocks of 128 rows
        dmp.gemm_wgrad8(dmp.quant8(torch.zeros(6, 20, device="cuda"), block=128), y)
    with pytest.raises(ValueError):  # groups of operands
        dmp.gemm_wgrad8(dmp.quant8(torch.zeros(2, 6, 20, device="cuda")), y)
    with pytest.raises(ValueError):
        dmp.gemm_wgrad8(x, y, out=torch.zeros(20, 9, device="cuda"))
    with pytest.raises(ValueError):
        dmp.gemm_wgrad8(x, y, torch.tensor([0, 6], device="cuda"), out=torch.zeros(20, 8, device="cuda"))


def test_route(dmp):
    x = torch.zeros(5, 6, device="cuda")
    r = dmp.route(x, 2)
    for bad in (0, 7):
        with pytest.raises(ValueError):
            dmp.route(x, bad)
    for bad in (x[0], x[None], x.t(), torch.zeros(2, 1025, device="cuda"), torch.zeros(2, 0, device="cuda")):
        with pytest.raises(ValueError):
            dmp.route(bad, 2)
    with pytest.raises(ValueError):
        dmp.route(torch.zeros(2, 100, device="cuda"), 65)
    with pytest.raises(TypeError):
        dmp.route(x, 2, mask=torch.ones(5, device="cuda"))
    for bad in (torch.ones(4, dtype=torch.bool, device="cuda"), torch.ones(5, dtype=torch.bool),
                torch.ones(10, dtype=torch.bool, device="cuda")[::2]):
        with pytest.raises(ValueError):
            dmp.route(x, 2, mask=bad)
    with pytest.raises(TypeError):
        dmp.route_grad(r, torch.zeros(5, 2, dtype=torch.float64, device="cuda"))
    for bad in (torch.zeros(5, 3, device="cuda"), torch.zeros(2, 5, device="cuda").t(), torch.zeros(5, 2)):
        with pytest.raises(ValueError):
            dmp.route_grad(r, bad)
    for bad in (torch.zeros(5, 7, device="cuda"), torch.zeros(5, 6, dtype=torch.bfloat16, device="cuda"), torch.zeros(6, 5, device="cuda").t()):
        with pytest.raises(ValueError):
            dmp.route_grad(r, None, 0.1, out=bad)


def test_scratch_is_asked_for(dmp):
    """A call that needs scratch and gets none is refused."""
    h = dmp.default_handle()
    assert h.wgrad8_work(0, 1, 64, 128, 8192, 128) > 0 and h.wgrad8_work(0, 1, -1, 128, 8192, 128) == -1
    assert h.wgrad8_work(2, 1, 64, 128, 100, 128) == 100 * 128 * 2 and h.wgrad8_work(0, 1, 64, 128, 100, 128) == 0
    assert h.adapters_work(0, 0, 4, 4, 64, 64, 8, 64, 64, dmp.GEMM_OUT_BF16) > 0
    assert h.wgrad8_work(0, 1, 1 << 30, 1 << 30, 8, 1 << 30) == -1 and h.wgrad8_work(0, 1 << 16, 1 << 22, 1 << 22, 8, 1 << 22) == -1
    assert h.adapters_work(0, 0, 4, 4, 64, 64, 0, 64, 64, 0) == -1 and h.adapters_work(0, 0, 4, 4, 1 << 22, 64, 8, 64, 1 << 22, 0) == -1
    assert h.route_work(100, 8) > 0 and h.route_work(100, 1025) == -1
    x = dmp.quant8(torch.zeros(8192, 64, device="cuda"), pow2=True)
    y = torch.zeros(8192, 128, dtype=torch.bfloat16, device="cuda")
    d = torch.zeros(64, 128, device="cuda")
    assert h.run_wgrad8(x.operand, y.data_ptr(), 0, d.data_ptr(), 0, 1, 64, 128, 8192, 128, 128, dmp.GEMM_BF16) == 1
