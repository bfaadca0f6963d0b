"""An 8-bit operand that a program keeps and changes: gemm_scaled8 reads the tensors that
the operand holds at the call, not the addresses it was made with."""
import copy
import io

import pytest

from test_gpu_scaled8 import E4, E5, dmp  # noqa: F401

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def operands(dmp):  # noqa: F811
    g = torch.Generator(device="cuda").manual_seed(1)
    draw = lambda *s: torch.randint(-4, 5, s, generator=g, device="cuda").float()  # noqa: E731
    A = dmp.Scaled8(draw(70, 256).to(E4), torch.full((70, 2), 0.5, device="cuda"))
    B = dmp.Scaled8(draw(136, 256).to(E4), torch.full((2, 2), 2.0, device="cuda"), block=128)
    return A, B, A.q.float() @ B.q.float().t().contiguous()


def test_replaced_scales_and_values(dmp):  # noqa: F811
    A, B, want = operands(dmp)
    kept = A.scale, B.q  # (the old ones stay alive: reading them would go unnoticed otherwise)
    assert torch.equal(dmp.gemm_scaled8(A, B), want)
    A.scale = A.scale * 4
    assert torch.equal(dmp.gemm_scaled8(A, B), 4 * want)
    A.scale = A.scale.t().contiguous().t()  # other strides
    assert torch.equal(dmp.gemm_scaled8(A, B), 4 * want)
    B.q = (2 * B.q.float()).to(E5)  # another format
    assert torch.equal(dmp.gemm_scaled8(A, B), 8 * want)
    B.scale.mul_(2)  # in place
    assert torch.equal(dmp.gemm_scaled8(A, B), 16 * want)
    assert kept[0].shape == (70, 2) and kept[1].dtype == E4


def test_quantized_operand_with_other_scales(dmp):  # noqa: F811
    A, B, _ = operands(dmp)
    X = A.q.float()
    A = dmp.quant8(X)
    first = dmp.gemm_scaled8(A, B)
    A.scale = A.scale * 0.25
    assert torch.equal(dmp.gemm_scaled8(A, B), 0.25 * first)


def test_memory_that_moved(dmp):  # noqa: F811
    """Weights whose storage is given back and taken again elsewhere, as offloading does."""
    A, B, want = operands(dmp)
    host, storage = B.q.cpu(), B.q.untyped_storage()
    size, at = storage.nbytes(), B.q.data_ptr()
    storage.resize_(0)
    taken = torch.empty(size, dtype=torch.uint8, device="cuda")  # what lies there now
    storage.resize_(size)
    assert B.q.data_ptr() != at and taken.numel() == size
    B.q.copy_(host)
    assert torch.equal(dmp.gemm_scaled8(A, B), want)


def test_copies_and_saved_operands(dmp):  # noqa: F811
    A, B, _ = operands(dmp)
    for C in (B, dmp.quant8(B.q.float(), block=128)):
        first = dmp.gemm_scaled8(A, C)
        deep, shallow, file = copy.deepcopy(C), copy.copy(C), io.BytesIO()
        torch.save(C, file)
        file.seek(0)
        saved = torch.load(file, weights_only=False)  # written above
        assert deep.q.data_ptr() != C.q.data_ptr() and shallow.q is C.q
        C.scale.mul_(2)
        for other, factor in ((deep, 1), (saved, 1), (shallow, 2)):
            assert torch.equal(dmp.gemm_scaled8(A, other), factor * first)


def test_changes_that_do_not_fit_are_refused(dmp):  # noqa: F811
    for change in (lambda o: setattr(o, "q", o.q[:, :240]), lambda o: setattr(o, "scale", o.scale[:, :1]),
                   lambda o: setattr(o, "K", 200), lambda o: setattr(o, "block", 64),
                   lambda o: setattr(o, "q", o.q.cpu()), lambda o: setattr(o, "scale", o.scale.cpu())):
        A, B, _ = operands(dmp)
        change(A)
        with pytest.raises(ValueError):
            dmp.gemm_scaled8(A, B)
    A, B, _ = operands(dmp)
    B.scale = B.scale.half()
    with pytest.raises(TypeError):
        dmp.gemm_scaled8(A, B)
    A, B, want = operands(dmp)
    A.q = A.q[:50]  # rows and scales together
    A.scale = A.scale[:50]
    assert torch.equal(dmp.gemm_scaled8(A, B), want[:50])
