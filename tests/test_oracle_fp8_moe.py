"""Pins of the 8-bit and expert-layer oracles: e4m3 rounding against every value
of the format and torch's own conversion, hand-made blocks, and the expert layer
against a direct sum.  CPU only."""
import numpy as np
import torch

from oracle import fp8_oracle as F
from oracle import moe_oracle as M


def _all_e4m3():
    v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    return np.unique(v[np.isfinite(v)])


def test_rounding_keeps_every_value_and_halves_to_even():
    v = _all_e4m3()
    assert v.max() == 448.0 and len(v) == 253           # 254 finite codes, two of them zero
    assert np.array_equal(F.e4m3_round(v), v)
    mid = (v[1:] + v[:-1]) / 2
    got = F.e4m3_round(mid)
    want = torch.from_numpy(mid).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(got, want)


def test_rounding_matches_torch_on_random_values():
    g = np.random.default_rng(0)
    v = (g.standard_normal(20000) * np.exp(g.uniform(-9, 6, 20000))).astype(np.float32)
    v = v[np.abs(v) <= 448]
    assert np.array_equal(F.e4m3_round(v), torch.from_numpy(v).to(torch.float8_e4m3fn).double().numpy())


def test_hand_block():
    x = np.zeros((1, 130), np.float32)
    x[0, 0], x[0, 1], x[0, 129] = 896.0, -1.0, 7.0
    q, s = F.quantize(x, 1, 128)
    assert s.tolist() == [[2.0, 7.0 / 448.0]]
    assert q[0, 0] == 448.0 and q[0, 1] == -0.5 and q[0, 129] == 448.0 and q[0, 2] == 0.0


def test_zero_block_has_a_small_finite_scale():
    q, s = F.quantize(np.zeros((3, 16), np.float32), 1, 128)
    assert not q.any() and np.all(s > 0) and np.all(np.isfinite(s))


def test_select_order_and_ties():
    s = np.array([[0.5, 0.9, 0.5, 0.7, 0.5]], np.float32)
    z = np.zeros(5, np.float32)
    assert M.select(s, z, 3).tolist() == [[1, 3, 0]]
    assert M.select(s, z, 2).tolist() == [[1, 3]]
    assert M.select(s, np.array([0, 0, 1, 0, 0], np.float32), 2).tolist() == [[2, 1]]


def test_experts_against_a_direct_sum():
    g = np.random.default_rng(1)
    x, wg, wu, wd = (g.standard_normal(s) for s in ((2, 3), (4, 5, 3), (4, 5, 3), (4, 3, 5)))
    idx, p = np.array([[0, 2], [3, 2]]), np.array([[0.4, 0.6], [0.1, 0.9]])
    want = np.zeros((2, 3))
    for t in range(2):
        for j in range(2):
            e = idx[t, j]
            for n in range(5):
                a = sum(x[t, i] * wg[e, n, i] for i in range(3))
                b = sum(x[t, i] * wu[e, n, i] for i in range(3))
                want[t] += p[t, j] * a / (1 + np.exp(-a)) * b * wd[e, :, n]
    assert np.allclose(M.experts(x, wg, wu, wd, idx, p)[0], want, rtol=1e-12, atol=1e-12)
