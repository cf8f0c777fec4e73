"""The autograd linear layer on tensors as autograd and callers hand them over."""
import pytest
import torch

import group_sparse_swiglu_amd as E
from gpu_common import DEV, note, require_gpu

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _rand(*shape, dtype=BF, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)


def _off(t):
    """t's values in a contiguous tensor one element past an aligned address."""
    flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    flat[1:] = t.flatten()
    u = flat[1:].view(t.shape)
    assert u.is_contiguous() and u.data_ptr() % 16
    return u


def test_without_gradients():
    require_gpu()
    note("linear no_grad")
    x, w = _rand(7, 5, 144), torch.nn.Parameter(_rand(32, 144, dtype=F32, seed=1))
    y = E.fp8_linear(x, w)
    for mode in (torch.no_grad, torch.inference_mode):
        with mode():
            assert torch.equal(E.fp8_linear(x, w), y)
            assert E.fp8_linear(x[0, 0], w).shape == (32,) and E.fp8_linear(x[:0], w).shape == (0, 5, 32)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_unaligned_tensors(dtype):
    require_gpu()
    note(f"linear unaligned {dtype}")
    x, w, dy = _rand(37, 144, dtype=dtype), _rand(32, 144, dtype=F32, seed=1), _rand(37, 32, dtype=dtype, seed=2)
    want = torch.autograd.grad(E.fp8_linear(x.requires_grad_(), w.requires_grad_()), (x, w), dy)
    xo, wo = _off(x.detach()).requires_grad_(), _off(w.detach()).requires_grad_()
    y = E.fp8_linear(xo, wo)
    assert torch.equal(y, E.fp8_linear(x, w))
    got = torch.autograd.grad(y, (xo, wo), _off(dy))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # a gradient that autograd itself cuts from a flat buffer
    y = E.fp8_linear(x, w)
    flat = torch.cat([torch.zeros(3, dtype=dtype, device=DEV), y.flatten()])
    got = torch.autograd.grad(flat, (x, w), torch.cat([torch.ones(3, dtype=dtype, device=DEV), dy.flatten()]))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
