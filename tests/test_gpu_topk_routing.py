"""GPU parity of the routing with groups, softmax scores and a gradient against the
fp64 oracle.  The choice is defined by keys that are rounded the same everywhere, so
indices are compared for equality, ties included.  Scores are off by at most 2^-20
of themselves (and 2^-125), weights by twice that and a few roundings: 2^-18.  A
logit's gradient is a product of a score, its complement, and a difference whose
terms are off by 2^-17 of their |sum|, rounded to its type."""
import numpy as np
import pytest
import torch

import group_sparse_swiglu_amd as E
from gpu_common import DEV, f64, note, require_gpu
from oracle import expert_block_oracle as O

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _logits(T, E_, dtype, kind, seed):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(T, E_, generator=g)
    if kind == "ties":          # few distinct logits
        z = torch.randint(-2, 3, (T, E_), generator=g).float()
    if kind == "near":          # neighbouring float32 values
        z = 1.0 + torch.randint(0, 4, (T, E_), generator=g) * 2.0 ** -23
    if kind == "wide":          # saturated scores, scores below float32's normal range
        z = z * 60
    if kind == "masked":
        z = z.masked_fill(torch.rand(T, E_, generator=g) < 0.7, float("-inf"))
        z[0] = float("-inf")
    return z.to(dtype)


def _check(z, k, scoring, bias, groups, keep, normalize, scaling, seed=0):
    zn = f64(z)
    want = O.route(zn, k, scoring, None if bias is None else bias.numpy(), groups, keep)
    args = dict(scoring=scoring, expert_bias=None if bias is None else bias.to(DEV), groups=groups, topk_groups=keep,
                normalize=normalize, scaling_factor=scaling)
    zd = z.to(DEV).requires_grad_()
    p, idx = E.topk_routing(zd, k, **args)
    assert idx.dtype == torch.int32 and np.array_equal(idx.cpu().numpy(), want)
    c = 1.0 if scaling is None else scaling
    wp = O.weights(zn, want, scoring, normalize, c)
    tiny = 2.0 ** -120 * (1e20 if normalize else 1)
    assert (np.abs(f64(p) - wp) <= 2.0 ** -18 * np.abs(wp) + tiny).all()
    dp = torch.randn(p.shape, generator=torch.Generator().manual_seed(seed + 9))
    (dz,) = torch.autograd.grad(p, zd, dp.to(DEV))
    wz, mag = O.weights_backward(f64(dp), zn, want, scoring, normalize, c)
    out = 2.0 ** -8 if z.dtype == BF else 2.0 ** -24
    assert dz.dtype == z.dtype
    assert (np.abs(f64(dz) - wz) <= out * np.abs(wz) + 2.0 ** -17 * mag + tiny).all()


SHAPES = [(1, 1, 1, 1, 1), (5, 2, 1, 1, 1), (37, 43, 11, 1, 1), (64, 256, 8, 8, 4), (9, 16, 16, 1, 1), (33, 60, 6, 6, 2),
          (17, 6, 2, 6, 3), (21, 384, 12, 6, 3), (19, 1024, 32, 1, 1), (7, 320, 20, 64, 5), (130, 257, 5, 1, 1),
          (11, 1000, 9, 1, 1), (13, 512, 32, 32, 3), (10, 48, 4, 3, 2), (6, 130, 3, 65, 65)]


@pytest.mark.parametrize("kind", ["normal", "ties", "near", "wide", "masked"])
@pytest.mark.parametrize("T,E_,k,groups,keep", SHAPES)
def test_choice_weights_gradient(T, E_, k, groups, keep, kind):
    require_gpu()
    for i, (scoring, dtype) in enumerate((s, d) for s in ("softmax", "sigmoid") for d in (F32, BF)):
        for biased in (False, True):
            note(f"route T={T} E={E_} k={k} groups={groups}/{keep} {kind} {scoring} {dtype} bias={biased}")
            z = _logits(T, E_, dtype, kind, T + E_ + i)
            g = torch.Generator().manual_seed(3)
            bias = (torch.rand(E_, generator=g) - 0.5) * (0.2 if scoring == "sigmoid" else 2 / E_) if biased else None
            if biased and kind == "ties":
                bias = torch.round(bias * 8) / 8
            _check(z, k, scoring, bias, groups, keep, normalize=(i + biased) % 2 == 0, scaling=2.5 if biased else None, seed=i)


def test_many_rows_and_strided_bias():
    require_gpu()
    note("route 3001 x 256, strided bias")
    z = _logits(3001, 256, BF, "normal", 1)
    store = torch.zeros(256, 3, device=DEV)
    bias = 0.1 * torch.rand(256, generator=torch.Generator().manual_seed(2))
    store[:, 1] = bias.to(DEV)
    p, idx = E.topk_routing(z.to(DEV), 8, "sigmoid", store[:, 1], 8, 4)
    p2, idx2 = E.topk_routing(z.to(DEV), 8, "sigmoid", bias.to(DEV), 8, 4)
    assert torch.equal(idx, idx2) and torch.equal(p, p2)
    assert np.array_equal(idx.cpu().numpy(), O.route(f64(z), 8, "sigmoid", bias.numpy(), 8, 4))
    one = E.topk_routing(z[1777:1778].to(DEV), 8, "sigmoid", bias.to(DEV), 8, 4)
    assert torch.equal(one[0], p[1777:1778]) and torch.equal(one[1], idx[1777:1778])


def test_agrees_with_sigmoid_topk_routing():
    require_gpu()
    note("route against sigmoid_topk_routing")
    z = _logits(500, 256, F32, "normal", 4).to(DEV)
    bias = (0.1 * torch.rand(256, generator=torch.Generator().manual_seed(2))).to(DEV)
    p, idx = E.topk_routing(z, 8, "sigmoid", bias, scaling_factor=2.5)
    q, order = E.sigmoid_topk_routing(z, bias, 8, scaling_factor=2.5)
    by = order.argsort(1)
    assert torch.equal(order.gather(1, by).int(), idx)
    assert torch.allclose(q.gather(1, by), p, rtol=2.0 ** -17)


def test_non_finite_rows():
    require_gpu()
    note("route non-finite")
    z = torch.randn(6, 40, generator=torch.Generator().manual_seed(0))
    z[1, 3] = float("nan")
    z[2, 5] = float("inf")
    z[3] = float("nan")
    z[4, :38] = float("-inf")
    clean = E.topk_routing(z[[0, 5]].to(DEV), 4, "softmax")
    for scoring in ("softmax", "sigmoid"):
        p, idx = E.topk_routing(z.to(DEV), 4, scoring)
        i = idx.cpu().numpy()
        assert (i >= 0).all() and (i < 40).all() and all(len(set(r)) == 4 and list(r) == sorted(r) for r in i)
        assert torch.isnan(p[1]).all() and torch.isnan(p[3]).all() and torch.isfinite(p[[0, 4, 5]]).all()
        assert torch.isnan(p[2]).all() if scoring == "softmax" else (torch.isfinite(p[2]).all() and 5 in i[2])
        assert 3 not in i[1] and {38, 39} <= set(i[4])
    p, idx = E.topk_routing(z.to(DEV), 4, "softmax")
    assert torch.equal(p[[0, 5]], clean[0]) and torch.equal(idx[[0, 5]], clean[1])
    bias = torch.zeros(40)
    bias[7], bias[8] = float("nan"), float("inf")
    _, idx = E.topk_routing(z[[0, 5]].to(DEV), 4, "sigmoid", bias.to(DEV))
    assert (idx == 8).any(1).all() and not (idx == 7).any()


def test_backward_skips_bad_indices_and_empty_batches():
    require_gpu()
    note("route bad indices, empty")
    z = torch.randn(3, 20, device=DEV)
    idx = torch.tensor([[0, 5, 20], [-1, 2, 3], [1, 2, 2 ** 31 - 1]], dtype=torch.int32, device=DEV)
    dz = E.topk_routing_bwd(torch.ones(3, 3, device=DEV), z, idx, "sigmoid", normalize=False)
    s = torch.sigmoid(z.double())
    want = torch.zeros_like(s)
    for t, j in ((0, 0), (0, 5), (1, 2), (1, 3), (2, 1), (2, 2)):
        want[t, j] = s[t, j] * (1 - s[t, j])
    assert torch.allclose(dz.double(), want, rtol=1e-5, atol=1e-12)
    e = torch.empty(0, 20, device=DEV, requires_grad=True)
    p, i = E.topk_routing(e, 3)
    assert p.shape == (0, 3) and i.shape == (0, 3)
    (g,) = torch.autograd.grad(p, e, torch.empty(0, 3, device=DEV))
    assert g.shape == e.shape


def test_unaligned_rows():
    require_gpu()
    note("route unaligned")
    flat = torch.randn(1 + 64 * 256, generator=torch.Generator().manual_seed(0))
    for dtype in (F32, BF):
        z = flat.to(dtype).to(DEV)[1:].view(64, 256)   # rows at 4 or 2 bytes past a 16-byte boundary
        a, b = E.topk_routing(z, 8, "softmax", groups=8, topk_groups=3), E.topk_routing(z.clone(), 8, "softmax", groups=8,
                                                                                         topk_groups=3)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        d = torch.randn(64, 8, device=DEV)
        assert torch.equal(E.topk_routing_bwd(d, z, a[1]), E.topk_routing_bwd(d, z.clone(), a[1]))


@pytest.mark.parametrize("gap", [10.0, 22.0, 40.0, 45.0, 60.0])
def test_chosen_scores_far_below_one(gap):
    """The expert that holds the softmax is kept out by its bias: the chosen ones' sum is e^-gap, down to 1e-20 and below."""
    require_gpu()
    for E_, k in ((12, 3), (256, 8), (600, 5)):
        note(f"route chosen scores of e^-{gap}, {E_} experts")
        z = torch.randn(40, E_, generator=torch.Generator().manual_seed(E_))
        z[:, 3] = gap + 3.0
        bias = torch.zeros(E_)
        bias[3] = -5.0
        zn = f64(z)
        idx = torch.stack([torch.randperm(E_ - 4, generator=torch.Generator().manual_seed(t))[:k].sort().values + 4 for t in range(40)]).int()
        assert 3 not in E.topk_routing(z.to(DEV), k, "softmax", bias.to(DEV))[1]
        dp = torch.randn(40, k, generator=torch.Generator().manual_seed(9))
        dz = E.topk_routing_bwd(dp.to(DEV), z.to(DEV), idx.to(DEV), "softmax", True, 2.5)
        wz, mag = O.weights_backward(f64(dp), zn, idx.numpy(), "softmax", True, 2.5)
        assert (np.abs(f64(dz) - wz) <= 2.0 ** -24 * np.abs(wz) + 2.0 ** -17 * (mag + np.abs(wz)) + 2.0 ** -53).all()


def test_expanded_gradients_and_no_second_derivative():
    require_gpu()
    note("route expanded gradients, second derivatives refused")
    z = _logits(9, 60, F32, "normal", 1)
    zd = z.to(DEV).requires_grad_()
    p, idx = E.topk_routing(zd, 6, "sigmoid", normalize=False)
    g, = torch.autograd.grad(p, zd, torch.ones(1, 1, device=DEV).expand(p.shape).requires_grad_(), create_graph=True)  # stride 0
    wz, mag = O.weights_backward(np.ones(p.shape), f64(z), idx.cpu().numpy(), "sigmoid", False, 1.0)
    assert (np.abs(f64(g) - wz) <= 2.0 ** -17 * mag).all()
    with pytest.raises(RuntimeError, match="once_differentiable|differentiat"):
        torch.autograd.grad(g.sum(), zd)
