"""GPU parity of the whole expert layer for a few tokens against the fp64 oracle.

Tolerances: a logit is a float32 sum over d of exact products, so it is within
(d/32 + 16) 2^-24 of its sum of |terms|; a probability moves by at most that
(the slope of log sigmoid is below one), twice for the normalisation, plus a
few float32 roundings.  y: half a unit of bf16 (2^-8 |y| with room) plus 2^-12 of
the sum of its |terms| for the float32 sums under h (their error is relative to
the terms before cancellation), the exponential and h's 16 bits."""
import numpy as np
import pytest
import torch

import group_sparse_swiglu_amd as E
from gpu_common import DEV, f64, note, require_gpu
from oracle import fp8_oracle as F
from oracle import moe_oracle as O

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _inputs(T, Ex, d, ff, seed, weights="bf16"):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, d, generator=g) * torch.exp(0.5 * torch.randn(d, generator=g))).to(BF)
    r = (torch.randn(Ex, d, generator=g) * d ** -0.5).to(BF)
    b = 0.1 * torch.rand(Ex, generator=g) - 0.05
    ws = [(torch.randn(Ex, *s, generator=g) * s[1] ** -0.5).to(BF) for s in ((ff, d), (ff, d), (d, ff))]
    return x, r, b, ws


def _run(x, r, b, ws, k, scaling, weights, **kw):
    dev = [w.to(DEV) for w in ws]
    vals, scales = [f64(w) for w in ws], None
    if weights == "fp8":
        pairs = [E.fp8_quantize_weight(w) for w in dev]
        dev, scales = [p[0] for p in pairs], tuple(p[1] for p in pairs)
        vals = [np.stack([F.values(q, s, 128, 128) for q, s in zip(f64(p[0]), p[1].cpu().numpy())]) for p in pairs]
    got = E.moe_decode(x.to(DEV), r.to(DEV), b.to(DEV), *dev, k, scaling_factor=scaling, scales=scales, **kw)
    return got, vals, (dev, scales)


def _compare(x, r, b, vals, k, scaling, got):
    y, p, idx = got
    xs = f64(x)
    z, mag = O.logits(xs, f64(r))
    score = 1.0 / (1.0 + np.exp(-z))
    tol = (x.shape[1] / 32 + 16) * 2.0 ** -24 * mag.max(axis=1)
    ref = O.select(score.astype(np.float32), b.numpy(), k)
    gi = idx.cpu().numpy()
    key = np.sort(score + f64(b), axis=1)[:, ::-1]
    # rows whose k-th and k+1-th (and k-1-th: order) keys are clearly apart choose, and order, the same
    gap = np.full(len(key), np.inf)
    for other in (k, k - 2):
        if 0 <= other < key.shape[1] and other != k - 1:
            gap = np.minimum(gap, np.abs(key[:, k - 1] - key[:, other]))
    clear = gap > 2 * tol + 2.0 ** -22
    assert clear.mean() > 0.9 or len(clear) < 16
    assert np.array_equal(gi[clear], ref[clear])
    assert all(len(set(row)) == k and row.min() >= 0 and row.max() < key.shape[1] for row in gi)
    rp = O.probs(score, gi, scaling)
    assert np.all(np.abs(f64(p) - rp) <= rp * (2 * tol[:, None] + 2.0 ** -20))
    ry, ymag = O.experts(xs, *vals, gi, rp)
    err, bound = np.abs(f64(y) - ry), 2.0 ** -8 * np.abs(ry) + 2.0 ** -12 * ymag
    assert np.all(err <= bound), f"error {np.max(err / bound):.2f} of the bound"


# tokens, experts, k, d, ff: one of everything, ragged K chunks, more tokens than one, two, four tiles on one expert
CASES = [(1, 1, 1, 16, 16), (1, 8, 2, 64, 48), (1, 256, 8, 256, 128), (2, 16, 16, 80, 144), (3, 43, 11, 272, 128),
         (15, 8, 3, 144, 32), (16, 64, 6, 128, 176), (17, 5, 2, 1040, 64), (31, 300, 8, 64, 64), (33, 4, 1, 128, 400),
         (48, 1024, 32, 32, 16), (64, 2, 2, 256, 80), (64, 256, 8, 144, 48), (64, 1, 1, 528, 272)]


@pytest.mark.parametrize("weights", ["bf16", "fp8"])
@pytest.mark.parametrize("T,Ex,k,d,ff", CASES)
def test_layer_matches_oracle(T, Ex, k, d, ff, weights):
    require_gpu()
    note(f"moe {T} {Ex} {k} {d} {ff} {weights}")
    x, r, b, ws = _inputs(T, Ex, d, ff, T + Ex)
    scaling = 2.5 if T % 2 else None
    got, vals, (dev, scales) = _run(x, r, b, ws, k, scaling, weights)
    _compare(x, r, b, vals, k, scaling, got)
    again = E.moe_decode(x.to(DEV), r.to(DEV), b.to(DEV), *dev, k, scaling_factor=scaling, scales=scales)
    assert all(torch.equal(a, c) for a, c in zip(again, got))


# more than 16 tokens with an odd number of 16-column tiles of y, more experts than 256, parts of y by either count
MANY = [(20, 12, 3, 272, 144), (64, 40, 6, 784, 400), (33, 300, 4, 48, 272), (17, 1, 1, 16, 16), (64, 64, 6, 1040, 272)]


@pytest.mark.parametrize("weights", ["bf16", "fp8"])
@pytest.mark.parametrize("T,Ex,k,d,ff", MANY)
def test_many_tokens(T, Ex, k, d, ff, weights):
    test_layer_matches_oracle(T, Ex, k, d, ff, weights)


@pytest.mark.parametrize("weights", ["bf16", "fp8"])
def test_wide_layer(weights):
    require_gpu()
    note(f"moe wide {weights}")
    x, r, b, ws = _inputs(6, 12, 2048, 1408, 5)
    got, vals, _ = _run(x, r, b, ws, 4, 1.0, weights)
    _compare(x, r, b, vals, 4, 1.0, got)


def test_routing_agrees_with_the_routing_call():
    """The same scores through sigmoid_topk_routing: d = 16 and small integers make the logits exact."""
    require_gpu()
    note("moe routing")
    g = torch.Generator().manual_seed(3)
    x = torch.randint(-3, 4, (64, 16), generator=g).to(BF)
    r = torch.randint(-2, 3, (96, 16), generator=g).to(BF) / 8
    b = (torch.randint(0, 3, (96,), generator=g) / 16).float()       # few distinct keys: many ties
    w = torch.zeros(96, 16, 16, dtype=BF, device=DEV)
    for k in (1, 8, 32):
        _, p, i = E.moe_decode(x.to(DEV), r.to(DEV), b.to(DEV), w, w, w, k, scaling_factor=2.5)
        logits = (x.float() @ r.float().t()).to(DEV)
        p2, i2 = E.sigmoid_topk_routing(logits, b.to(DEV), k, 2.5)
        assert torch.equal(i, i2) and torch.equal(p, p2)


def test_strided_bias_given_outputs_and_zero_tokens():
    require_gpu()
    note("moe strided bias")
    x, r, b, ws = _inputs(4, 16, 64, 32, 9)
    got, vals, (dev, _) = _run(x, r, b, ws, 3, None, "bf16")
    wide = torch.zeros(16, 3)
    wide[:, 1] = b
    out = tuple(torch.full_like(t, 77) for t in got)
    ws_dict = {}
    for _ in range(2):
        res = E.moe_decode(x.to(DEV), r.to(DEV), wide.to(DEV)[:, 1], *dev, 3, out=out, workspace=ws_dict)
        assert all(a is c for a, c in zip(res, out)) and all(torch.equal(a, c) for a, c in zip(out, got))
    y, p, i = E.moe_decode(x[:0].to(DEV), r.to(DEV), b.to(DEV), *dev, 3)
    assert y.shape == (0, 64) and p.shape == (0, 3) and i.shape == (0, 3)


@pytest.mark.parametrize("weights", ["bf16", "fp8"])
def test_non_finite_values_stay_where_they_belong(weights):
    """Infinite and NaN weights of an expert reach only the tokens that chose it;
    a NaN token reaches no other."""
    require_gpu()
    note(f"moe non-finite {weights}")
    T, Ex, d, ff, k = 20, 8, 256, 64, 2
    x, r, b, ws = _inputs(T, Ex, d, ff, 21)
    (y, p, idx), _, (dev, scales) = _run(x, r, b, ws, k, None, weights)
    hit = (idx == 3).any(dim=1)
    assert 0 < int(hit.sum()) < T
    bad = [w.clone() for w in dev]
    for w in bad:
        if weights == "bf16":
            w[3, 5, 7], w[3, 0, 0] = float("nan"), float("inf")
        else:
            w.view(torch.uint8)[3, 5, 7] = 0x7f          # NaN of e4m3
    y2, p2, i2 = E.moe_decode(x.to(DEV), r.to(DEV), b.to(DEV), *bad, k, scales=scales)
    assert torch.equal(i2, idx) and torch.equal(p2, p) and torch.equal(y2[~hit], y[~hit])
    assert torch.isnan(y2[hit]).any(dim=1).all()
    xn = x.clone()
    xn[4] = float("nan")
    y3, p3, i3 = E.moe_decode(xn.to(DEV), r.to(DEV), b.to(DEV), *dev, k, scales=scales)
    keep = torch.arange(T, device=DEV) != 4
    assert torch.equal(y3[keep], y[keep]) and torch.equal(i3[keep], idx[keep])
    assert torch.isnan(y3[4]).all() and int(i3[4].min()) >= 0 and int(i3[4].max()) < Ex and len(set(i3[4].tolist())) == k


def test_experts_past_32_bit_offsets():
    """Weights of more than 2^32 bytes each: the bias sends every token to the last experts."""
    require_gpu()
    note("moe past 2^32")
    Ex, ff, d, k = 260, 4096, 2064, 2
    g = torch.Generator(device=DEV).manual_seed(1)
    ws = [torch.empty(Ex, *s, dtype=BF, device=DEV) for s in ((ff, d), (ff, d), (d, ff))]
    for w in ws:
        w[:-2].zero_()
        w[-2:] = torch.randn(2, *w.shape[1:], device=DEV, generator=g) * w.shape[2] ** -0.5
    x, r, b, _ = _inputs(3, Ex, d, 16, 2)
    b[-2:] += 2.0
    got = E.moe_decode(x.to(DEV), r.to(DEV), b.to(DEV), *ws, k)
    assert sorted(set(got[2].flatten().tolist())) == [Ex - 2, Ex - 1]
    small = [f64(w[-2:]) for w in ws]
    vals = [lambda e, s=s: s[e - (Ex - 2)] for s in small]
    _compare(x, r, b, vals, k, None, got)


def test_on_another_stream_and_in_a_graph():
    require_gpu()
    note("moe graph")
    x, r, b, ws = _inputs(5, 64, 256, 128, 33)
    dev = [t.to(DEV) for t in (x, r, b, *ws)]
    work = {}
    want = E.moe_decode(*dev, 6, workspace=work)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = E.moe_decode(*dev, 6, workspace=work)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, c) for a, c in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = E.moe_decode(*dev, 6, workspace=work)
    for seed in (1, 2, 3):
        dev[0].copy_(_inputs(5, 64, 256, 128, seed)[0].to(DEV))
        graph.replay()
        torch.cuda.synchronize()
        eager = E.moe_decode(*dev, 6)
        assert all(torch.equal(a, c) for a, c in zip(out, eager))


@pytest.mark.parametrize("weights", ["bf16", "fp8"])
def test_workgroups_that_do_not_wait_give_the_same(weights):
    """Without patience a workgroup computes the gate/up units it misses itself."""
    require_gpu()
    for T, Ex, k, d, ff in ((1, 256, 8, 1024, 512), (40, 32, 4, 512, 272)):
        note(f"moe patience {T} {weights}")
        x, r, b, ws = _inputs(T, Ex, d, ff, 7)
        got, _, (dev, scales) = _run(x, r, b, ws, k, None, weights)
        try:
            for polls in (0, 1, 3):
                E.moe_decode_set_patience(polls)
                again = E.moe_decode(x.to(DEV), r.to(DEV), b.to(DEV), *dev, k, scales=scales)
                assert all(torch.equal(a, c) for a, c in zip(again, got))
        finally:
            E.moe_decode_set_patience()


def test_concurrent_calls_on_two_streams():
    require_gpu()
    note("moe two streams")
    x, r, b, ws = _inputs(8, 64, 2048, 512, 11)
    got, _, (dev, _) = _run(x, r, b, ws, 8, None, "bf16")
    args = (x.to(DEV), r.to(DEV), b.to(DEV), *dev, 8)
    streams, outs = [torch.cuda.Stream() for _ in range(3)], []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(E.moe_decode(*args))
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, c) for a, c in zip(o, got))


def test_arguments_are_refused():
    require_gpu()
    x, r, b, ws = _inputs(4, 8, 64, 32, 1)
    dev = [w.to(DEV) for w in ws]
    xd, rd, bd = x.to(DEV), r.to(DEV), b.to(DEV)
    with pytest.raises(E.EsgError):
        E.moe_decode(xd.float(), rd, bd, *dev, 2)
    with pytest.raises(E.EsgError):
        E.moe_decode(xd, rd.float(), bd, *dev, 2)
    with pytest.raises(E.EsgError):
        E.moe_decode(xd, rd, b, *dev, 2)
    with pytest.raises(E.EsgError):
        E.moe_decode(xd, rd, bd, dev[0], dev[1].transpose(1, 2).contiguous().transpose(1, 2), dev[2], 2)
    with pytest.raises(E.EsgError):
        E.moe_decode(xd, rd, bd, *dev, 9)
    with pytest.raises(E.EsgError):
        E.moe_decode(xd.repeat(17, 1), rd, bd, *dev, 2)
    with pytest.raises(E.EsgError):
        E.moe_decode(xd, rd, bd, *dev, 2, out=(torch.empty(3, 64, dtype=BF, device=DEV),
                                               torch.empty(4, 2, device=DEV),
                                               torch.empty(4, 2, dtype=torch.int64, device=DEV)))
