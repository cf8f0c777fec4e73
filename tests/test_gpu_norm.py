"""GPU parity of the norm with the residual's addition against the fp64 oracle.

With u = 2^-24, one float32 rounding.  The sum of squares of a row adds at most 64
terms per lane and 9 levels over the lanes, all positive, so r is off by at most
(64 + 9) / 2 + 4 < 41 u of itself, and the float32 y by 44 u.  dx = dh + r (g - h r^2
mean(g h)): mean(g h) is off by 80 u of mean |g h|, r^3 by 123 u, a few roundings
more: at most 220 u of the sum of its |terms|.  dw: at most T additions and 46 u.  A
bf16 result adds its rounding, 2^-8 of the value."""
import numpy as np
import pytest
import torch

import group_sparse_swiglu_amd as E
from gpu_common import DEV, f64, note, require_gpu
from oracle import expert_block_oracle as O
from oracle import fp8_oracle as O8

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
EPS = 1e-5


def _rand(rows, cols, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp(0.7 * torch.randn(cols, generator=g))
    return (x * scale).to(dtype)


def _out(dtype):
    return 2.0 ** -8 if dtype == BF else U


def _case(T, d, dtype, wdtype, residual, seed):
    x = _rand(T, d, dtype, seed)
    res = _rand(T, d, dtype, seed + 1, 3.0) if residual else None
    w = (1 + 0.3 * torch.randn(d, generator=torch.Generator().manual_seed(seed + 2))).to(wdtype)
    h = x if res is None else (x.float() + res.float()).to(dtype)
    return x, res, w, h


SHAPES = [(1, 16), (3, 48), (5, 512), (7, 528), (4, 768), (9, 1024), (2, 1040), (33, 2048), (3, 2064), (5, 4096), (2, 5504),
          (3, 8192), (2, 8208), (2, 16384)]


@pytest.mark.parametrize("dtype,wdtype", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("T,d", SHAPES)
def test_forward_and_backward(T, d, dtype, wdtype):
    require_gpu()
    for residual in (True, False):
        note(f"norm {T}x{d} {dtype} {wdtype} residual={residual}")
        x, res, w, h = _case(T, d, dtype, wdtype, residual, T + d)
        xd, wd = x.to(DEV).requires_grad_(), w.to(DEV).requires_grad_()
        rd = res.to(DEV).requires_grad_() if residual else None
        out = E.rms_norm(xd, wd, rd, eps=EPS)
        y = out[0] if residual else out
        if residual:
            assert torch.equal(out[1].cpu(), h)
        want, r = O.rms_norm(f64(h), f64(w), EPS)
        assert y.dtype == dtype
        assert (np.abs(f64(y) - want) <= (_out(dtype) + 45 * U) * np.abs(want)).all()
        dy, dh = _rand(T, d, dtype, 5), _rand(T, d, dtype, 6) if residual else None
        if residual:
            gx, gr, gw = torch.autograd.grad(out, (xd, rd, wd), (dy.to(DEV), dh.to(DEV)))
            assert torch.equal(gx, gr)
        else:
            gx, gw = torch.autograd.grad(out, (xd, wd), dy.to(DEV))
        dx, dw, mx, mw = O.rms_norm_backward(f64(dy), f64(h), f64(w), EPS, None if dh is None else f64(dh))
        assert gx.dtype == dtype and gw.dtype == wdtype
        assert (np.abs(f64(gx) - dx) <= _out(dtype) * np.abs(dx) + 225 * U * mx).all()
        assert (np.abs(f64(gw) - dw) <= _out(wdtype) * np.abs(dw) + (T + 48) * U * mw).all()


@pytest.mark.parametrize("T,d", [(1500, 256), (5000, 2048)])
def test_many_rows(T, d):
    """More rows than workgroups, more workgroups than a weight gradient's parts."""
    require_gpu()
    note(f"norm {T}x{d}")
    x, res, w, h = _case(T, d, BF, F32, True, 1)
    y, hd, rstd = E.rms_norm_fwd(x.to(DEV), w.to(DEV), res.to(DEV), EPS)
    want, r = O.rms_norm(f64(h), f64(w), EPS)
    assert torch.equal(hd.cpu(), h)
    assert (np.abs(f64(rstd) - r[:, 0]) <= 41 * U * r[:, 0]).all()
    assert (np.abs(f64(y) - want) <= (2.0 ** -8 + 45 * U) * np.abs(want)).all()
    dy = _rand(T, d, BF, 5)
    dx, dw, mx, mw = O.rms_norm_backward(f64(dy), f64(h), f64(w), EPS)
    ws = {}
    gx, gw = E.rms_norm_bwd(dy.to(DEV), hd, w.to(DEV), rstd, workspace=ws)
    assert (np.abs(f64(gx) - dx) <= 2.0 ** -8 * np.abs(dx) + 225 * U * mx).all()
    assert (np.abs(f64(gw) - dw) <= (T + 48) * U * mw).all()
    g2, none = E.rms_norm_bwd(dy.to(DEV), hd, w.to(DEV), rstd, need_dw=False)
    assert none is None and torch.equal(gx, g2)
    g3, w3 = E.rms_norm_bwd(dy.to(DEV), hd, w.to(DEV), rstd, workspace=ws)
    assert torch.equal(gx, g3) and torch.equal(gw, w3)


def test_row_is_independent_of_the_batch():
    require_gpu()
    for d in (512, 2048, 8192):
        note(f"norm batch invariance {d}")
        x, _, w, _ = _case(3000, d, BF, BF, False, 2)
        xd, wd = x.to(DEV), w.to(DEV)
        y = E.rms_norm(xd, wd)
        assert torch.equal(E.rms_norm(xd[1234:1235].contiguous(), wd), y[1234:1235])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,d", [(1, 16), (3, 144), (5, 528), (64, 2048), (3, 5504), (2, 16384), (4100, 1024)])
def test_eight_bit_output(T, d, dtype):
    require_gpu()
    for residual in (True, False):
        note(f"norm fp8 {T}x{d} {dtype} residual={residual}")
        x, res, w, h = _case(T, d, dtype, F32, residual, T + d)
        got = E.rms_norm_quantize(x.to(DEV), w.to(DEV), None if res is None else res.to(DEV), EPS)
        if residual:
            assert torch.equal(got[2].cpu(), h)
        y, _ = O.rms_norm(f64(h), f64(w), EPS)
        q, s = f64(got[0]), got[1].cpu().numpy().astype(np.float64)
        assert got[0].dtype == torch.float8_e4m3fn and s.shape == (T, -(-d // 128))
        top = np.stack([np.abs(y[:, i:i + 128]).max(1) for i in range(0, d, 128)], 1)
        assert (np.abs(s - top / 448) <= 48 * U * s).all()
        v = q * np.repeat(s, 128, 1)[:, :d]
        unit = np.repeat(s, 128, 1)[:, :d]
        # half a step of e4m3: 2^-4 of the value, at least 2^-10 units
        assert (np.abs(v - y) <= np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10 * unit) + 100 * U * np.abs(y)).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,d", [(1, 32), (3, 160), (64, 2048), (3, 5504), (2, 16384), (4100, 768)])
def test_four_bit_output(T, d, dtype):
    require_gpu()
    note(f"norm mxfp4 {T}x{d} {dtype}")
    x, res, w, h = _case(T, d, dtype, BF, True, T + d)
    q, s, hd = E.rms_norm_quantize(x.to(DEV), w.to(DEV), res.to(DEV), EPS, format="mxfp4")
    assert torch.equal(hd.cpu(), h)
    y, _ = O.rms_norm(f64(h), f64(w), EPS)
    top = np.abs(y).reshape(T, d // 32, 32).max(-1)
    e = s.cpu().numpy().astype(np.int64)
    lo, hi = (np.floor(np.log2(top * (1 + k * 48 * U))) + 125 for k in (-1, 1))
    assert ((e == lo) | (e == hi)).all()
    v = O.mx_values(q.cpu().numpy(), s.cpu().numpy())
    unit = np.repeat(2.0 ** (e - 127.0), 32, 1)
    a = np.abs(y) / unit
    half = np.where(a < 2, 0.25, np.where(a < 4, 0.5, 1.0))
    near = np.abs(v - y) <= (half + 8 * 48 * U) * unit
    assert (near | ((a > 6) & (np.abs(v) == 6 * unit))).all() and (v * y >= 0).all()


def test_in_place_and_empty_and_shapes():
    require_gpu()
    note("norm in place, empty, leading shapes")
    x, res, w, h = _case(6, 768, BF, F32, True, 9)
    want_y, want_h, _ = E.rms_norm_fwd(x.to(DEV), w.to(DEV), res.to(DEV), EPS)
    xd, rd = x.to(DEV), res.to(DEV)
    y, hd, _ = E.rms_norm_fwd(xd, w.to(DEV), rd, EPS, out=xd, residual_out=rd)
    assert y is xd and hd is rd and torch.equal(y, want_y) and torch.equal(hd, want_h)
    xd, rd = x.to(DEV), res.to(DEV)
    q, s, hd = E.rms_norm_quantize(xd, w.to(DEV), rd, EPS, residual_out=xd)
    assert torch.equal(hd, want_h)
    y3 = E.rms_norm(x.to(DEV).view(2, 3, 768), w.to(DEV), eps=EPS)
    assert y3.shape == (2, 3, 768)
    assert torch.equal(y3.view(6, 768), E.rms_norm(x.to(DEV), w.to(DEV), eps=EPS))
    strided = x.to(DEV).t().contiguous().t()  # a copy is made of it
    assert torch.equal(E.rms_norm(strided, w.to(DEV), eps=EPS), y3.view(6, 768))
    shifted = torch.empty(6 * 768 + 1, dtype=BF, device=DEV)[1:].view(6, 768).copy_(x)  # not 16-byte aligned: copied
    assert torch.equal(E.rms_norm(shifted, w.to(DEV), eps=EPS), y3.view(6, 768))
    e = torch.empty(0, 768, dtype=BF, device=DEV, requires_grad=True)
    wd = w.to(DEV).requires_grad_()
    y0 = E.rms_norm(e, wd)
    gx, gw = torch.autograd.grad(y0, (e, wd), torch.empty_like(y0))
    assert gx.shape == e.shape and not gw.any()


def test_unused_outputs_and_frozen_weight():
    require_gpu()
    note("norm partial gradients")
    x, res, w, h = _case(5, 256, F32, F32, True, 3)
    dy = _rand(5, 256, F32, 5).to(DEV)
    xd, rd, wd = x.to(DEV).requires_grad_(), res.to(DEV).requires_grad_(), w.to(DEV)
    y, hd = E.rms_norm(xd, wd, rd, EPS)
    gx, = torch.autograd.grad(y, xd, dy, retain_graph=True)          # the new residual unused, the weight frozen
    dx, _, mx, _ = O.rms_norm_backward(f64(dy), f64(h), f64(w), EPS)
    assert (np.abs(f64(gx) - dx) <= 226 * U * mx).all()
    g2, = torch.autograd.grad(hd, rd, dy)                             # y unused
    assert torch.equal(g2, dy)
    wd = w.to(DEV).requires_grad_()
    y, hd = E.rms_norm(x.to(DEV), wd, res.to(DEV), EPS)
    gw, = torch.autograd.grad(y, wd, dy)                              # only the weight
    _, dw, _, mw = O.rms_norm_backward(f64(dy), f64(h), f64(w), EPS)
    assert (np.abs(f64(gw) - dw) <= 54 * U * mw).all()


def test_zero_and_large_rows():
    require_gpu()
    note("norm zero row, large row, NaN row")
    x = torch.zeros(4, 512)
    x[1] = 1e18
    x[2, 7] = float("nan")
    x[3] = 1.0
    y = E.rms_norm(x.to(DEV), torch.ones(512, device=DEV), eps=EPS).cpu()
    assert not y[0].any() and torch.allclose(y[1], torch.ones(512)) and torch.isnan(y[2]).all()
    assert torch.allclose(y[3], torch.ones(512), rtol=1e-5)
    q, s = E.rms_norm_quantize(x.to(DEV), torch.ones(512, device=DEV), eps=EPS, format="mxfp4")
    assert (s[2] == 255).all() and (s[0] == 0).all() and not q[0].any()


def test_gradient_of_large_values():
    """h of 2^100: its products with the gradient leave float32's range unless r comes first."""
    require_gpu()
    note("norm gradient of large values")
    for d in (512, 2048):
        x = _rand(4, d, F32, 1).double() * 2.0 ** 100
        w, dy = _rand(1, d, F32, 2)[0], _rand(4, d, F32, 3, 2.0 ** 40)
        xd, wd = x.float().to(DEV).requires_grad_(), w.to(DEV).requires_grad_()
        gx, gw = torch.autograd.grad(E.rms_norm(xd, wd, eps=EPS), (xd, wd), dy.to(DEV))
        dx, dw, mx, mw = O.rms_norm_backward(f64(dy), x.numpy(), f64(w), EPS)
        assert (np.abs(f64(gx) - dx) <= 226 * U * mx).all()
        assert (np.abs(f64(gw) - dw) <= 53 * U * mw).all()


@pytest.mark.parametrize("T", [15, 31, 33, 257, 1023, 1024, 1025])
def test_weight_gradient_around_the_change_of_kernels(T):
    require_gpu()
    for d, dtype, wdtype in ((16, F32, BF), (80, BF, F32), (1040, BF, BF), (2064, F32, F32)):
        note(f"norm weight gradient {T}x{d} {dtype} {wdtype}")
        x, _, w, _ = _case(T, d, dtype, wdtype, False, T)
        dy = _rand(T, d, dtype, 5)
        xd = x.to(DEV)
        _, h, r = E.rms_norm_fwd(xd, w.to(DEV), eps=EPS)
        gx, gw = E.rms_norm_bwd(dy.to(DEV), h, w.to(DEV), r)
        dx, dw, mx, mw = O.rms_norm_backward(f64(dy), f64(x), f64(w), EPS)
        assert (np.abs(f64(gx) - dx) <= _out(dtype) * np.abs(dx) + 225 * U * mx).all()
        assert (np.abs(f64(gw) - dw) <= _out(wdtype) * np.abs(dw) + (T + 48) * U * mw).all()
        again = E.rms_norm_bwd(dy.to(DEV), h, w.to(DEV), r)
        assert torch.equal(gx, again[0]) and torch.equal(gw, again[1])
        assert torch.equal(gx, E.rms_norm_bwd(dy.to(DEV), h, w.to(DEV), r, need_dw=False)[0])


def test_expanded_gradients_and_no_second_derivative():
    require_gpu()
    note("norm expanded gradients, second derivatives refused")
    x, res, w, h = _case(6, 528, F32, BF, True, 3)
    xd, rd, wd = (t.to(DEV).requires_grad_() for t in (x, res, w))
    y, hd = E.rms_norm(xd, wd, rd, EPS)
    gx, gw = torch.autograd.grad(y.sum() + 2 * hd.sum(), (xd, wd))     # gradients of stride 0
    dx, dw, mx, mw = O.rms_norm_backward(np.ones(h.shape), f64(h), f64(w), EPS, 2 * np.ones(h.shape))
    assert (np.abs(f64(gx) - dx) <= 226 * U * mx).all() and (np.abs(f64(gw) - dw) <= 2.0 ** -8 * np.abs(dw) + 55 * U * mw).all()
    y, _ = E.rms_norm(xd, wd, rd, EPS)
    g, = torch.autograd.grad(y, xd, torch.ones_like(y).requires_grad_(), create_graph=True)
    assert torch.equal(g, torch.autograd.grad(E.rms_norm(xd, wd, rd, EPS)[0].sum(), xd)[0])
    with pytest.raises(RuntimeError, match="once_differentiable|differentiat"):
        torch.autograd.grad(g.sum(), xd)
    with torch.autograd.set_multithreading_enabled(False):             # the backward on this thread
        y, _ = E.rms_norm(xd, wd, rd, EPS)
        assert torch.equal(torch.autograd.grad(y.sum() + 0 * y.sum(), xd)[0], g)
