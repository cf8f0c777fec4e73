"""What fp8_linear asks of its forward and backward calls.  CPU only: the calls
are stood in for by plain products that record their arguments."""
import pytest
import torch

import group_sparse_swiglu_amd as E


@pytest.fixture
def calls(monkeypatch):
    seen = []

    def fwd(x, w, need_dx=True, need_dw=True, workspace=None, out=None):
        seen.append(("fwd", need_dx, need_dw, x, w))
        saved = torch.cat([x.detach().flatten(), w.detach().flatten()]) if need_dx or need_dw else None
        return x.detach() @ w.detach().t().to(x.dtype), saved

    def bwd(dy, saved, d_in, w_dtype, need_dx=True, need_dw=True, workspace=None):
        seen.append(("bwd", need_dx, need_dw, dy))
        T = dy.shape[0]
        x, w = saved[: T * d_in].view(T, d_in), saved[T * d_in:].view(-1, d_in)
        return dy @ w if need_dx else None, (dy.t() @ x).to(w_dtype) if need_dw else None

    monkeypatch.setattr(E, "fp8_linear_fwd", fwd)
    monkeypatch.setattr(E, "fp8_linear_bwd", bwd)
    return seen


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
def test_nothing_is_kept_without_gradients(calls, mode):
    x, w = torch.randn(2, 3, 32), torch.nn.Parameter(torch.randn(16, 32))
    with mode():
        y = E.fp8_linear(x, w)
    assert y.shape == (2, 3, 16) and not y.requires_grad
    assert [c[:3] for c in calls] == [("fwd", False, False)]
    assert torch.equal(y, E.fp8_linear(x, w).detach())
    assert [c[:3] for c in calls] == [("fwd", False, False), ("fwd", False, True)]


def _off(*shape):
    """A contiguous tensor one element past an aligned address."""
    n = torch.Size(shape).numel()
    t = torch.randn(n + 1)[1:].view(shape)
    assert t.is_contiguous() and t.data_ptr() % 16
    return t


def test_tensors_at_unaligned_addresses_are_copied(calls):
    x, w, dy = _off(5, 32), _off(16, 32), _off(5, 16)
    y = E.fp8_linear(x.requires_grad_(), w.requires_grad_())
    dx, dw = torch.autograd.grad(y, (x, w), dy)
    with torch.no_grad():
        E.fp8_linear(x, w)
    assert len(calls) == 3
    for c in calls:
        for t in c[3:]:
            assert t.data_ptr() % 16 == 0 and t.is_contiguous()
    assert torch.allclose(dx, dy @ w) and torch.allclose(dw, dy.t() @ x)


def test_aligned_tensors_are_not_copied(calls):
    x, w, dy = torch.randn(5, 32), torch.randn(16, 32), torch.randn(5, 16)
    y = E.fp8_linear(x, w.requires_grad_())
    torch.autograd.grad(y, w, dy)
    assert [t.data_ptr() for c in calls for t in c[3:]] == [x.data_ptr(), w.data_ptr(), dy.data_ptr()]
