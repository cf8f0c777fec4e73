"""The expert block's oracle against values and identities outside itself: torch's
autograd and differences for the gradients, the 4-bit table, hand-made choices."""
import numpy as np
import pytest
import torch

from oracle import expert_block_oracle as O


def test_norm_gradient_is_autograd_and_differences():
    rng = np.random.default_rng(0)
    h, dy, dh = (rng.standard_normal((5, 32)) for _ in range(3))
    w = 1 + 0.3 * rng.standard_normal(32)
    th, tw = torch.tensor(h, requires_grad=True), torch.tensor(w, requires_grad=True)
    y = th * torch.rsqrt((th * th).mean(1, keepdim=True) + 1e-3) * tw
    assert np.allclose(y.detach().numpy(), O.rms_norm(h, w, 1e-3)[0], rtol=1e-13)
    gx, gw = torch.autograd.grad((y, th * 1.0), (th, tw), (torch.tensor(dy), torch.tensor(dh)))
    dx, dw, mx, mw = O.rms_norm_backward(dy, h, w, 1e-3, dh)
    assert np.allclose(gx.numpy(), dx, rtol=1e-11, atol=1e-13) and np.allclose(gw.numpy(), dw, rtol=1e-11, atol=1e-13)
    assert (np.abs(dx) <= mx * (1 + 1e-12)).all() and (np.abs(dw) <= mw * (1 + 1e-12)).all()
    loss = lambda a: np.sum(O.rms_norm(a, w, 1e-3)[0] * dy) + np.sum(a * dh)
    for i, j in ((0, 0), (3, 17), (4, 31)):
        e = np.zeros_like(h)
        e[i, j] = 1e-6
        assert abs((loss(h + e) - loss(h - e)) / 2e-6 - dx[i, j]) < 1e-7


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_routing_gradient_is_autograd_and_differences(scoring, normalize):
    rng = np.random.default_rng(1)
    z, dp = rng.standard_normal((6, 12)), rng.standard_normal((6, 4))
    idx = O.route(z, 4, scoring)
    t = torch.tensor(z, requires_grad=True)
    s = torch.softmax(t, 1) if scoring == "softmax" else torch.sigmoid(t)
    sel = s.gather(1, torch.tensor(idx))
    p = 1.5 * (sel / (sel.sum(1, keepdim=True) + 1e-20) if normalize else sel)
    assert np.allclose(p.detach().numpy(), O.weights(z, idx, scoring, normalize, 1.5), rtol=1e-13)
    (g,) = torch.autograd.grad(p, t, torch.tensor(dp))
    dz, mag = O.weights_backward(dp, z, idx, scoring, normalize, 1.5)
    assert np.allclose(g.numpy(), dz, rtol=1e-10, atol=1e-14) and (np.abs(dz) <= mag * (1 + 1e-9) + 1e-16).all()
    loss = lambda a: np.sum(O.weights(a, idx, scoring, normalize, 1.5) * dp)
    for i, j in ((0, 0), (5, 11)):
        e = np.zeros_like(z)
        e[i, j] = 1e-6
        assert abs((loss(z + e) - loss(z - e)) / 2e-6 - dz[i, j]) < 1e-7


def test_choices_by_hand():
    z = np.array([[3.0, 1.0, 2.0, 2.0, 0.0, 5.0]])
    assert O.route(z, 2, "softmax").tolist() == [[0, 5]]
    assert O.route(z, 3, "sigmoid").tolist() == [[0, 2, 5]]                       # 2 and 3 tie: the lower
    # groups of two: sums of the keys 3+1, 2+2, 0+5 in sigmoid's terms: .953+.731, .881+.881, .5+.993
    assert O.route(z, 2, "sigmoid", groups=3, topk_groups=1).tolist() == [[2, 3]]
    assert O.route(z, 2, "sigmoid", bias=np.array([0, 0, 0, 0, 0.9, 0.0]), groups=3, topk_groups=1).tolist() == [[4, 5]]
    assert O.route(np.full((1, 4), -np.inf), 2, "softmax").tolist() == [[0, 1]]
    assert O.weights(np.full((1, 4), -np.inf), np.array([[0, 1]]), "softmax", True, 1.0).tolist() == [[0.0, 0.0]]


def test_four_bit_table():
    u = np.array([0.0, 0.25, 0.26, 0.75, 0.74, 1.25, 1.75, 2.5, 2.51, 3.5, 5.0, 5.01, 7.9, -0.0, -3.0])
    assert O.e2m1(u).tolist() == [0, 0, 1, 2, 1, 2, 4, 4, 5, 6, 6, 7, 7, 8, 13]
    x = np.zeros((1, 64), np.float32)
    x[0, :3] = [7.0, -1.0, 0.3]           # exponent of 7 is 2: unit 1
    x[0, 32:34] = [2.0 ** -149, 0.0]      # far below: byte 0, unit 2^-127
    codes, e = O.mx_quantize(x)
    assert e.tolist() == [[127, 0]] and codes[0, :3].tolist() == [7, 10, 1] and not codes[0, 32:].any()
    v = O.mx_values(O.mx_pack(codes), e)
    assert v[0, :3].tolist() == [6.0, -1.0, 0.5]
