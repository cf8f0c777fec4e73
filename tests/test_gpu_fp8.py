"""GPU parity of the 8-bit block-scaled operators against the fp64 oracle.

Quantisation is defined to the bit and compared so.  Tolerances of the product
(KB blocks of 128 along K, mag = the sum of the |terms| of an output):
- float32 results: each of the KB block sums adds a few float32 roundings (four
  chained products, scale, FMA), so |error| <= (KB + 32) 2^-24 mag;
- bfloat16 results: half a unit of bfloat16, 2^-8 |y| with room for the sum's own
  error, plus 2^-13 mag for what the 8-bit products drop (at most 2^-13.7 of mag
  was measured for single products)."""
import numpy as np
import pytest
import torch

import group_sparse_swiglu_amd as E
from gpu_common import DEV, f64, note, require_gpu
from oracle import fp8_oracle as O

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _x(rows, cols, dtype, seed, kind="normal"):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp(0.7 * torch.randn(cols, generator=g))
    if kind == "wide":      # from subnormals of float32 to large values, whole blocks of zeros
        x = torch.sign(x) * torch.exp2(torch.randint(-140, 100, (rows, cols), generator=g).float())
        x[:, : min(cols, 128)] = 0
    if kind == "ties":      # few distinct significands: many products next to a tie of e4m3
        x = torch.randint(-255, 256, (rows, cols), generator=g).float()
    return x.to(dtype)


def _same(q, scale, want_q, want_s):
    assert np.array_equal(f64(q), want_q)
    assert np.array_equal(scale.cpu().numpy(), want_s)


QUANT = [(1, 16), (1, 128), (3, 144), (128, 128), (129, 272), (37, 2048), (300, 1040), (16, 5504), (255, 400)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", QUANT)
def test_quantize_rows_and_columns(rows, cols, dtype):
    require_gpu()
    for kind in ("normal", "wide", "ties"):
        note(f"quant {rows}x{cols} {dtype} {kind}")
        x = _x(rows, cols, dtype, rows + cols, kind)
        xd = x.to(DEV)
        want = O.quantize(x.float().numpy(), 1, 128)
        _same(*E.fp8_quantize(xd), *want)
        q, s, qt, st = E.fp8_quantize(xd, transposed=True)
        _same(q, s, *want)
        qw, sw = O.quantize(x.float().numpy().T, 1, 128)
        assert qt.shape == (cols, (rows + 15) // 16 * 16) and st.shape == (cols, (rows + 127) // 128)
        assert np.array_equal(f64(qt)[:, :rows], qw) and not f64(qt)[:, rows:].any()
        assert np.array_equal(st.cpu().numpy(), sw)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("batch,rows,cols", [(None, 128, 128), (None, 1, 16), (None, 129, 144), (3, 40, 272), (2, 300, 128)])
def test_quantize_tiles(batch, rows, cols, dtype):
    require_gpu()
    note(f"quant tiles {batch} {rows}x{cols} {dtype}")
    shape = (rows, cols) if batch is None else (batch, rows, cols)
    w = _x((batch or 1) * rows, cols, dtype, 7).view(shape)
    q, s, qt, st = E.fp8_quantize_weight(w.to(DEV), transposed=True)
    q2, s2 = E.fp8_quantize_weight(w.to(DEV))
    assert torch.equal(q2.view(torch.uint8), q.view(torch.uint8)) and torch.equal(s, s2)
    for b in range(batch or 1):
        at = (lambda t: t) if batch is None else (lambda t: t[b])
        qw, sw = O.quantize(at(w).float().numpy(), 128, 128)
        _same(at(q), at(s), qw, sw)
        assert np.array_equal(f64(at(qt))[:, :rows], qw.T) and not f64(at(qt))[:, rows:].any()
        assert np.array_equal(at(st).cpu().numpy(), sw.T)


def test_quantize_non_finite_blocks_only():
    require_gpu()
    note("quant non-finite")
    x = _x(140, 400, F32, 3)
    x[2, 5], x[130, 200] = float("inf"), float("nan")
    q, s, qt, st = E.fp8_quantize(x.to(DEV), transposed=True)
    row = torch.isfinite(s.cpu())
    assert (~row).nonzero().tolist() == [[2, 0], [130, 1]]
    col = torch.isfinite(st.cpu())
    assert (~col).nonzero().tolist() == [[5, 0], [200, 1]]
    clean = x.clone()
    clean[2, 5] = clean[130, 200] = 0.0
    qc, sc = O.quantize(clean.numpy(), 1, 128)
    keep = np.repeat(row.numpy(), 128, 1)[:, :400]
    assert np.array_equal(f64(q)[keep], qc[keep]) and np.array_equal(s.cpu().numpy()[row.numpy()], sc[row.numpy()])
    # a product with such a block is NaN, the other rows are untouched
    w = E.fp8_quantize_weight(_x(64, 400, F32, 4).to(DEV))
    y = E.fp8_matmul(q, s, *w, out_dtype=F32)
    assert torch.isnan(y[2]).all() and torch.isnan(y[130]).all()
    assert torch.isfinite(y).all(dim=1).sum() == 138


def _check(y, av, bv, out, KB):
    ref, mag = av @ bv.T, np.abs(av) @ np.abs(bv).T
    err = np.abs(f64(y) - ref)
    tol = (KB + 32) * 2.0 ** -24 * mag if out == F32 else 2.0 ** -8 * np.abs(ref) + 2.0 ** -13 * mag
    assert np.all(err <= tol + 1e-37), f"error {np.max(err / np.maximum(tol, 1e-37)):.2f} of the bound"


# few rows, one tile, ragged tiles, one K block and less, several tiles, split K, large tiles
MATMUL = [(1, 16, 16), (1, 1, 128), (2, 130, 144), (5, 300, 2048), (16, 2048, 5504), (17, 257, 400), (33, 129, 1040),
          (64, 512, 1280), (65, 100, 272), (100, 128, 16), (128, 128, 8208), (129, 255, 2064), (200, 77, 1024),
          (300, 1030, 640), (257, 131, 4112), (511, 640, 768)]


@pytest.mark.parametrize("form", ["tiles", "rows"])
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("M,N,K", MATMUL)
def test_matmul(M, N, K, out, form):
    require_gpu()
    note(f"matmul {M}x{N}x{K} {form} {out}")
    a = E.fp8_quantize(_x(M, K, BF, 1).to(DEV))
    b = (E.fp8_quantize_weight if form == "tiles" else E.fp8_quantize)(_x(N, K, F32, 2).to(DEV))
    y = E.fp8_matmul(*a, *b, out_dtype=out)
    av = O.values(f64(a[0]), a[1].cpu().numpy(), 1, 128)
    bv = O.values(f64(b[0]), b[1].cpu().numpy(), 128 if form == "tiles" else 1, 128)
    _check(y, av, bv, out, (K + 127) // 128)
    assert torch.equal(E.fp8_matmul(*a, *b, out_dtype=out).view(torch.uint8), y.view(torch.uint8))


# chunks of 64 rows, one to many; K split over workgroups, into uneven parts and with a partial last block; the
# smallest products that the tile kernel takes, ragged, with and without a split
MATMUL_ROUTES = [(70, 16, 144), (130, 2050, 400), (448, 100, 5136), (1025, 33, 272), (4096, 16, 128), (3, 40, 16400),
                 (64, 513, 4112), (48, 64, 30000), (127, 129, 12304), (70, 4111, 144), (2000, 300, 176),
                 (300, 1700, 2064), (1100, 777, 4240)]


@pytest.mark.parametrize("form", ["tiles", "rows"])
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("M,N,K", MATMUL_ROUTES)
def test_matmul_routes(M, N, K, out, form):
    test_matmul(M, N, K, out, form)


@pytest.mark.parametrize("form", ["tiles", "rows"])
@pytest.mark.parametrize("out", [BF, F32])
def test_matmul_large_tiles_sampled(out, form):
    """Enough 256 x 256 tiles to fill the card, ragged on both sides; every
    output against float64 on the device (itself checked on 64 rows against the CPU)."""
    require_gpu()
    M, N, K = 4133, 4366, 784
    note(f"matmul large {form} {out}")
    a = E.fp8_quantize(_x(M, K, BF, 5).to(DEV))
    b = (E.fp8_quantize_weight if form == "tiles" else E.fp8_quantize)(_x(N, K, BF, 6).to(DEV))
    y = E.fp8_matmul(*a, *b, out_dtype=out)
    av = O.values(f64(a[0]), a[1].cpu().numpy(), 1, 128)
    bv = O.values(f64(b[0]), b[1].cpu().numpy(), 128 if form == "tiles" else 1, 128)
    rows = np.unique(np.concatenate([np.arange(0, M, 97), [255, 256, 4095, 4096, M - 1]]))
    _check(y[torch.from_numpy(rows).to(DEV)], av[rows], bv, out, 7)
    A, B = torch.from_numpy(av).to(DEV), torch.from_numpy(bv).to(DEV)
    ref, mag = A @ B.t().contiguous(), A.abs() @ B.t().abs().contiguous()
    tol = (7 + 32) * 2.0 ** -24 * mag if out == F32 else 2.0 ** -8 * ref.abs() + 2.0 ** -13 * mag
    assert bool(((y.double() - ref).abs() <= tol).all())


def test_matmul_past_32_bit_offsets():
    """a of more than 2^31 bytes, results past 2^31 elements: the last rows."""
    require_gpu()
    note("matmul past 2^31")
    M, N, K = 2_200_000, 1040, 1024
    a = torch.empty(M, K, dtype=torch.uint8, device=DEV)
    tail = E.fp8_quantize(_x(300, K, BF, 8).to(DEV))
    a.zero_()
    a[-300:] = tail[0].view(torch.uint8)
    sa = torch.ones(M, 8, device=DEV)
    sa[-300:] = tail[1]
    b = E.fp8_quantize_weight(_x(N, K, BF, 9).to(DEV))
    y = E.fp8_matmul(a.view(torch.float8_e4m3fn), sa, *b)
    _check(y[-300:], O.values(f64(tail[0]), tail[1].cpu().numpy(), 1, 128),
           O.values(f64(b[0]), b[1].cpu().numpy(), 128, 128), BF, 8)
    assert not y[:1000].any() and not y[-1300:-300].any()


def test_quantize_past_32_bit_offsets():
    require_gpu()
    note("quant past 2^31")
    x = torch.zeros(1_100_000, 2048, dtype=BF, device=DEV)
    tail = _x(260, 2048, BF, 10)
    x[-260:] = tail.to(DEV)
    q, s = E.fp8_quantize(x)
    _same(q[-260:], s[-260:], *O.quantize(tail.float().numpy(), 1, 128))
    del q, s
    q, s, qt, st = E.fp8_quantize(x, transposed=True)
    _same(q[-260:], s[-260:], *O.quantize(tail.float().numpy(), 1, 128))
    first = 1_100_000 // 128 * 128          # the last, partial block of rows
    n = 1_100_000 - first
    qw, sw = O.quantize(tail.float().numpy()[-n:].T, 1, 128)
    assert np.array_equal(f64(qt[:, first:1_100_000]), qw) and np.array_equal(st[:, -1:].cpu().numpy(), sw)


def test_zero_sizes():
    require_gpu()
    note("fp8 zero sizes")
    q, s, qt, st = E.fp8_quantize(torch.empty(0, 256, dtype=BF, device=DEV), transposed=True)
    assert q.shape == (0, 256) and s.shape == (0, 2) and qt.shape == (256, 0) and st.shape == (256, 0)
    w = E.fp8_quantize_weight(_x(32, 256, BF, 1).to(DEV))
    assert E.fp8_matmul(q, s, *w).shape == (0, 32)
    x = torch.empty(0, 256, dtype=BF, device=DEV, requires_grad=True)
    wp = _x(32, 256, F32, 1).to(DEV).requires_grad_()
    y = E.fp8_linear(x, wp)
    dx, dw = torch.autograd.grad(y, (x, wp), torch.empty(0, 32, dtype=BF, device=DEV))
    assert dx.shape == (0, 256) and not dw.any()


def test_non_contiguous_and_mixed_arguments_are_refused():
    require_gpu()
    x = _x(64, 256, BF, 1).to(DEV)
    with pytest.raises(E.EsgError):
        E.fp8_quantize(x.t())
    with pytest.raises(E.EsgError):
        E.fp8_quantize(x[:, :128])
    q, s = E.fp8_quantize(x)
    with pytest.raises(E.EsgError):
        E.fp8_matmul(x, s, q, s)
    with pytest.raises(E.EsgError):
        E.fp8_matmul(q, s, q, s, out_dtype=torch.float16)
    with pytest.raises(E.EsgError):
        E.fp8_matmul(q, s.t().contiguous().t(), q, s)
    with pytest.raises(E.EsgError):
        E.fp8_matmul(q, s, q, s, out=torch.empty(64, 63, device=DEV))


@pytest.mark.parametrize("wdtype", [BF, F32])
@pytest.mark.parametrize("T,K,N", [(1, 128, 16), (5, 144, 272), (130, 256, 384), (333, 768, 2048), (1000, 272, 144)])
def test_linear_against_the_formula(T, K, N, wdtype):
    require_gpu()
    note(f"linear {T} {K} {N} {wdtype}")
    x, w, dy = _x(T, K, BF, 1), _x(N, K, wdtype, 2) * K ** -0.5, _x(T, N, BF, 3) * 1e-3
    xd, wd = x.to(DEV).requires_grad_(), w.to(DEV).requires_grad_()
    y = E.fp8_linear(xd, wd)
    dx, dw = torch.autograd.grad(y, (xd, wd), dy.to(DEV))
    assert y.dtype == BF and dx.dtype == BF and dw.dtype == wdtype
    outs, mags = O.linear(*(t.float().numpy() for t in (x, w, dy)))
    for got, ref, mag, KB in zip((y, dx, dw), outs, mags, ((K + 127) // 128, (N + 127) // 128, (T + 127) // 128)):
        tol = (KB + 32) * 2.0 ** -24 * mag if got.dtype == F32 else 2.0 ** -8 * np.abs(ref) + 2.0 ** -13 * mag
        assert np.all(np.abs(f64(got) - ref) <= tol + 1e-37)


def test_linear_gradient_against_differences():
    """Every block holds 448 or -448, so scales are 1 and integers up to 16 are
    kept exactly: the layer is then the exact bilinear map, and a difference of
    the loss over one changed entry is its gradient, in whole numbers."""
    require_gpu()
    note("linear differences")
    g = torch.Generator().manual_seed(0)
    T, K, N = 40, 160, 48

    def ints(r, c):
        t = torch.randint(-8, 9, (r, c), generator=g).float()
        t[::3, 0], t[1::3, 0], t[2::3, 0] = 448.0, -448.0, 448.0   # a maximum in every row block ...
        t[:, 128::128] = 448.0
        t[0, :] = 448.0                                            # ... and column block
        return t

    x, w, dy = ints(T, K), ints(N, K), ints(T, N)
    xd, wd = x.to(DEV).requires_grad_(), w.to(DEV).requires_grad_()
    y = E.fp8_linear(xd, wd)
    assert np.array_equal(f64(y), x.double().numpy() @ w.double().numpy().T)
    dx, dw = torch.autograd.grad(y, (xd, wd), dy.to(DEV))

    def loss(a, b):
        return (E.fp8_linear(a.to(DEV), b.to(DEV)).double() * dy.to(DEV).double()).sum().item()

    base = loss(x, w)
    for i, j in ((3, 5), (17, 100), (39, 159), (8, 127)):
        step = x.clone()
        step[i, j] += 1.0
        assert loss(step, w) - base == dx[i, j].item()
    for i, j in ((1, 3), (20, 90), (47, 159), (11, 126)):
        step = w.clone()
        step[i, j] -= 1.0
        assert base - loss(x, step) == dw[i, j].item()


def test_linear_single_gradients_and_leading_dims():
    require_gpu()
    note("linear partial gradients")
    x, w = _x(24, 128, BF, 1).to(DEV).view(2, 3, 4, 128), _x(32, 128, F32, 2).to(DEV)
    dy = _x(24, 32, BF, 3).to(DEV).view(2, 3, 4, 32)
    both = torch.autograd.grad(E.fp8_linear(x.requires_grad_(), w.requires_grad_()), (x, w), dy)
    assert both[0].shape == x.shape and both[1].shape == w.shape
    only_x = torch.autograd.grad(E.fp8_linear(x, w.detach()), x, dy)[0]
    only_w = torch.autograd.grad(E.fp8_linear(x.detach(), w), w, dy)[0]
    assert torch.equal(only_x, both[0]) and torch.equal(only_w, both[1])
    # a gradient that comes as an expanded or transposed view
    s = torch.autograd.grad(E.fp8_linear(x, w).sum(), x)[0]
    assert torch.equal(s, torch.autograd.grad(E.fp8_linear(x, w), x, torch.ones_like(dy))[0])


def test_linear_calls_agree_with_the_parts_and_autograd():
    require_gpu()
    note("linear calls")
    T, K, N = 200, 272, 144
    x, w, dy = _x(T, K, BF, 1).to(DEV), _x(N, K, F32, 2).to(DEV), _x(T, N, BF, 3).to(DEV)
    ws = {}
    y, saved = E.fp8_linear_fwd(x, w, workspace=ws)
    dx, dw = E.fp8_linear_bwd(dy, saved, K, F32, workspace=ws)
    xq, xs, xqt, xst = E.fp8_quantize(x, transposed=True)
    wq, wsc, wqt, wst = E.fp8_quantize_weight(w, transposed=True)
    dq, ds, dqt, dst = E.fp8_quantize(dy, transposed=True)
    assert torch.equal(y, E.fp8_matmul(xq, xs, wq, wsc))
    assert torch.equal(dx, E.fp8_matmul(dq, ds, wqt, wst))
    assert torch.equal(dw, E.fp8_matmul(dqt, dst, xqt, xst, out_dtype=F32))
    y2, none = E.fp8_linear_fwd(x, w, False, False, workspace=ws)
    assert none is None and torch.equal(y2, y)
    _, half = E.fp8_linear_fwd(x, w, True, False, workspace=ws)
    only = E.fp8_linear_bwd(dy, half, K, F32, True, False, workspace=ws)
    assert torch.equal(only[0], dx) and only[1] is None
    with pytest.raises(E.EsgError):
        E.fp8_linear_bwd(dy, half, K, F32, workspace=ws)      # saved without the weight gradient's part
    with pytest.raises(E.EsgError):
        E.fp8_linear_fwd(x, w[:, :256].contiguous())


def test_on_another_stream_and_in_a_graph():
    require_gpu()
    note("fp8 graph")
    M, N, K = 128, 128, 8208      # split K: two launches and a workspace
    x, w = _x(M, K, BF, 1).to(DEV), _x(N, K, BF, 2).to(DEV)
    ws = {}

    def step():
        q, s = E.fp8_quantize(x)
        b, sb = E.fp8_quantize_weight(w)
        return E.fp8_matmul(q, s, b, sb, out_dtype=F32, workspace=ws)

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
        step()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (3, 4, 5):
        x.copy_(_x(M, K, BF, seed).to(DEV))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, step())
