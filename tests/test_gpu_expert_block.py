"""The norm, the routing and the 4-bit products run together as a block of experts, eagerly,
as captured graphs and on several streams, and at offsets past 32 bits."""
import numpy as np
import pytest
import torch

import group_sparse_swiglu_amd as E
from gpu_common import DEV, f64, note, require_gpu
from oracle import expert_block_oracle as O

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-6


class Block:
    """A residual stream's norm, the router over the shared-bias groups, gate, up and down products in 4 bits."""

    def __init__(self, d, ff, experts, k, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.E, self.k = experts, k
        self.norm = (1 + 0.2 * torch.randn(d, generator=g)).to(DEV)
        self.router = (torch.randn(experts, d, generator=g) * d ** -0.5).to(BF).to(DEV)
        self.bias = (0.05 * torch.rand(experts, generator=g)).to(DEV)
        self.plain = [(torch.randn(experts, n, m, generator=g) * m ** -0.5).to(BF).to(DEV) for n, m in ((ff, d), (ff, d), (d, ff))]
        self.w = [E.mxfp4_quantize(w) for w in self.plain]
        self.ws = {}

    def __call__(self, x, residual):
        y, h, _ = E.rms_norm_fwd(x, self.norm, residual, EPS, need_rstd=False)
        q, s, _ = E.rms_norm_quantize(x, self.norm, residual, EPS, format="mxfp4")
        p, idx = E.topk_routing(y @ self.router.t(), self.k, "sigmoid", self.bias, 4, 2, True, 2.5)
        offsets, rows, inv = E.bucket_by_group(idx, self.E)
        gate, up = (E.mxfp4_grouped_matmul(q, s, *w, offsets, rows, workspace=self.ws) for w in self.w[:2])
        act = torch.nn.functional.silu(gate) * up
        down = E.mxfp4_grouped_matmul(*E.mxfp4_quantize(act), *self.w[2], offsets, workspace=self.ws)
        out = (down.float()[inv.long()] * p[..., None]).sum(1)
        return h, y, q, s, p, idx, offsets, rows, inv, gate, up, act, down, out


def _input(T, d, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(T, d, generator=g).to(BF).to(DEV) for _ in range(2)]


def _product(av, bv, got, K):
    want, mag = av @ bv.T, np.abs(av) @ np.abs(bv).T
    tol = (K / 128 + 24) * 2.0 ** -22 * mag + 2.0 ** -8 * np.abs(want)
    assert (np.abs(f64(got) - want) <= tol).all()


@pytest.mark.parametrize("T", [1, 5, 64, 700])
def test_block(T):
    """Every step against float64 from what it was given, the whole against the experts' weights before their rounding."""
    require_gpu()
    note(f"block of experts {T} tokens")
    d, ff, Ex, k = 512, 288, 16, 4
    block = Block(d, ff, Ex, k)
    x, res = _input(T, d, T)
    h, y, q, s, p, idx, offsets, rows, inv, gate, up, act, down, out = block(x, res)
    hn = (x.float() + res.float()).to(BF)
    assert torch.equal(h, hn)
    yn, _ = O.rms_norm(f64(hn), f64(block.norm), EPS)
    assert (np.abs(f64(y) - yn) <= (2.0 ** -8 + 2.0 ** -18) * np.abs(yn)).all()
    z = f64(y @ block.router.t())
    want = O.route(z, k, "sigmoid", block.bias.cpu().numpy(), 4, 2)
    assert np.array_equal(idx.cpu().numpy(), want)
    wp = O.weights(z, want, "sigmoid", True, 2.5)
    assert (np.abs(f64(p) - wp) <= 2.0 ** -18 * wp).all()
    off, rows_, inv_ = (t.cpu().numpy() for t in (offsets, rows, inv))
    assert off[-1] == T * k and np.array_equal(np.repeat(np.arange(Ex), np.diff(off))[inv_], want)
    av = O.mx_values(q.cpu().numpy(), s.cpu().numpy())[rows_]
    hq, hs = E.mxfp4_quantize(act)
    hv = O.mx_values(hq.cpu().numpy(), hs.cpu().numpy())
    ws = [O.mx_values(*(t.cpu().numpy() for t in w)) for w in block.w]
    for e in range(Ex):
        at = slice(off[e], off[e + 1])
        _product(av[at], ws[0][e], gate[at], d)
        _product(av[at], ws[1][e], up[at], d)
        _product(hv[at], ws[2][e], down[at], ff)
    o = (f64(down)[inv_] * f64(p)[..., None]).sum(1)
    mag = (np.abs(f64(down)[inv_]) * f64(p)[..., None]).sum(1)
    assert (np.abs(f64(out) - o) <= (k + 1) * 2.0 ** -24 * mag).all()
    # beside the unrounded experts: rounding to 4 bits moves a vector by a tenth or so at each of four places
    full = np.zeros_like(o)
    wg, wu, wd = (f64(w) for w in block.plain)
    for t in range(T):
        for j in range(k):
            e = want[t, j]
            a = wg[e] @ yn[t]
            full[t] += wp[t, j] * (wd[e] @ (a / (1 + np.exp(-a)) * (wu[e] @ yn[t])))
    assert np.linalg.norm(o - full) <= 0.4 * np.linalg.norm(full)


def test_block_as_a_graph():
    """One token and many: every replay is the eager call, with other work and new inputs between."""
    require_gpu()
    d, ff, Ex, k = 512, 288, 16, 4
    block = Block(d, ff, Ex, k)
    for T in (2, 300):
        note(f"block as a graph, {T} tokens")
        inputs = [_input(T, d, s) for s in (1, 2, 3, 1)]
        want = [[t.clone() for t in block(*i)] for i in inputs]
        x, res = (t.clone() for t in inputs[0])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            block(x, res)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = block(x, res)
        for i, w in zip(inputs, want):
            for t in out:
                t.zero_()
            x.copy_(i[0])
            res.copy_(i[1])
            other = block(*inputs[1])                  # beside the graph, with the same dict
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, w))
            assert all(torch.equal(a, b) for a, b in zip(other, want[1]))


def test_training_step_and_its_graph():
    """Gradients through norm, router and weights against float64; captured by the explicit calls and by autograd.

    Every one of the eight stages (norm, logits, routing, weighting, and back) adds at most d + 48 terms with float32
    roundings and its terms' norm is at most sqrt(d) = 16 times its value's: 8 * 304 * 16 * 2^-24 = 2.3e-3."""
    require_gpu()
    note("training step")
    T, d, Ex, k, cap = 200, 256, 24, 3, 1.5
    g = torch.Generator().manual_seed(4)
    x, res, dh = (torch.randn(T, d, generator=g) for _ in range(3))
    w, wr, val = 1 + 0.2 * torch.randn(d, generator=g), torch.randn(Ex, d, generator=g) * d ** -0.5, torch.randn(Ex, d, generator=g)
    leaves = [t.to(DEV).requires_grad_() for t in (x, res, w, wr, val)]
    dhd = dh.to(DEV)

    def loss(leaves):
        xd, rd, wd, wrd, vald = leaves
        y, h = E.rms_norm(xd, wd, rd, EPS)
        p, idx = E.topk_routing(y @ wrd.t(), k, "softmax", normalize=True, scaling_factor=cap)
        out = ((y @ vald.t()).gather(1, idx.long()) * p).sum()
        return out + (h * dhd).sum(), idx

    def step():
        value, idx = loss(leaves)
        return [*torch.autograd.grad(value, leaves), idx]

    *grads, idx = step()
    ref = [t.double().requires_grad_() for t in (x, res, w, wr, val)]
    h = ref[0] + ref[1]
    y = h * (h.pow(2).mean(1, keepdim=True) + EPS).rsqrt() * ref[2]
    zs = (y @ ref[3].t()).gather(1, idx.long().cpu()).softmax(1) * cap
    total = ((y @ ref[4].t()).gather(1, idx.long().cpu()) * zs).sum() + (h * dh.double()).sum()
    for a, b in zip(grads, torch.autograd.grad(total, ref)):
        assert (a.double().cpu() - b).norm() <= 2.3e-3 * b.norm()
    want = [t.clone() for t in (*grads, idx)]
    # no eager graph of the leaves lives here
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    note("training step captured")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    junk = torch.randn(1 << 20, device=DEV)
    for _ in range(3):
        for t in out:
            t.zero_()
        junk.mul_(1.0001).sum().item()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):  # gather's gradient adds in any order: at most k + 1 terms of each sum, times the above
            assert torch.equal(a, b) if a.dtype == torch.int32 else torch.allclose(a, b, rtol=1e-4, atol=1e-5)
    # the explicit calls, bit for bit
    xd, rd, wd = (t.detach() for t in leaves[:3])
    dy, z, dp = torch.randn(T, d, generator=g).to(DEV), torch.randn(T, Ex, generator=g).to(DEV), torch.randn(T, k, generator=g).to(DEV)
    ws = {}

    def calls():
        y, h, r = E.rms_norm_fwd(xd, wd, rd, EPS)
        p, i = E.topk_routing_fwd(z, k)
        return [y, h, r, p, i, *E.rms_norm_bwd(dy, h, wd, r, dhd, workspace=ws), E.topk_routing_bwd(dp, z, i)]

    want = [t.clone() for t in calls()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = calls()
    for _ in range(3):
        for t in out:
            t.zero_()
        calls()
        junk.mul_(1.0001).sum().item()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_streams_share_a_dict():
    """The operators that take scratch, side by side on three streams with one dict."""
    require_gpu()
    note("expert block on streams")
    cases, outs, cache = [], [], {}
    for i, (T, n) in enumerate(((3000, 512), (4100, 1040), (2000, 2048))):
        x, dy = _input(T, n, i)
        w = torch.ones(n, device=DEV)
        _, h, r = E.rms_norm_fwd(x, w)
        a, b = E.mxfp4_quantize(_input(5000 + 8 * i, 320 + 32 * i, i)[0]), E.mxfp4_quantize(_input(5400, 320 + 32 * i, i + 5)[0])
        be = [t.view(2, 2700, -1) for t in b]
        off = torch.tensor([0, 2000 + i, 4996], dtype=torch.int32, device=DEV)
        assert E.mxfp4_matmul_workspace_size(5000 + 8 * i, 5400, 320) > 0 < E.mxfp4_grouped_matmul_workspace_size(5000 + 8 * i, 2700, 320, 2)
        cases.append((lambda dy=dy, h=h, w=w, r=r: E.rms_norm_bwd(dy, h, w, r, workspace=cache),
                      lambda a=a, b=b: (E.mxfp4_matmul(*a, *b, workspace=cache),),
                      lambda a=a, be=be, off=off: (E.mxfp4_grouped_matmul(*a, *be, off, workspace=cache,
                                                                          out=torch.zeros(a[0].shape[0], 2700, device=DEV)),)))
    want = [[f() for f in c] for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(6):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs.append((i, [f() for f in cases[i]]))
    torch.cuda.synchronize()
    for i, got in outs:
        assert all(torch.equal(u, v) for g, w in zip(got, want[i]) for u, v in zip(g, w))


def test_a_graph_keeps_its_scratch_while_the_dict_grows():
    require_gpu()
    note("4-bit product: graph beside a growing dict")
    ops = [(E.mxfp4_quantize(_input(M, K, M)[0]), E.mxfp4_quantize(_input(4096, K, K)[0])) for M, K in ((4096, 1056), (6000, 2080))]
    assert all(E.mxfp4_matmul_workspace_size(M, 4096, K) > 0 for M, K in ((4096, 1056), (6000, 2080)))
    want = [E.mxfp4_matmul(*a, *b) for a, b in ops]
    cache = {}
    small = lambda: E.mxfp4_matmul(*ops[0][0], *ops[0][1], workspace=cache)  # noqa: E731
    small()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = small()
    for _ in range(3):
        out.zero_()
        got = E.mxfp4_matmul(*ops[1][0], *ops[1][1], workspace=cache)
        junk = [torch.full((1 << 18,), 7, dtype=torch.int32, device=DEV) for _ in range(4)]
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(got, want[1])
        del junk


def _last(t, n):
    return t[-n:].contiguous()


def test_offsets_past_32_bits_norm_and_values():
    """A row does not depend on the batch: the last rows of 2.3e9 elements are those of a small call."""
    require_gpu()
    note("norm past 32 bits")
    d, T = 16384, 140000
    x = torch.empty(T, d, dtype=BF, device=DEV)
    x.normal_(generator=torch.Generator(DEV).manual_seed(1))
    w = torch.ones(d, device=DEV)
    assert x.numel() > 2 ** 31
    small = _last(x, 3)
    y, h, r = E.rms_norm_fwd(x, w)
    assert torch.equal(y[-3:], E.rms_norm_fwd(small, w)[0])
    dx, dw = E.rms_norm_bwd(x, h, w, r)
    assert torch.equal(dx[-3:], E.rms_norm_bwd(small, small, w, _last(r, 3))[0]) and torch.isfinite(dw).all()
    del y, dx
    for fmt in ("fp8", "mxfp4"):
        q, s = E.rms_norm_quantize(x, w, format=fmt)
        qs, ss = E.rms_norm_quantize(small, w, format=fmt)
        assert torch.equal(q[-3:].view(torch.uint8), qs.view(torch.uint8)) and torch.equal(s[-3:], ss)
    note("4-bit values past 32 bits")
    q, s = E.mxfp4_quantize(x)
    qs, ss = E.mxfp4_quantize(small)
    assert torch.equal(q[-3:], qs) and torch.equal(s[-3:], ss)
    assert torch.equal(E.mxfp4_dequantize(q, s)[-3:], E.mxfp4_dequantize(qs, ss))


def test_offsets_past_32_bits_routing():
    require_gpu()
    note("routing past 32 bits")
    T, Ex, k = 2200000, 1024, 4
    z = torch.empty(T, Ex, dtype=BF, device=DEV)
    z.normal_(generator=torch.Generator(DEV).manual_seed(1))
    assert z.numel() > 2 ** 31
    p, i = E.topk_routing_fwd(z, k)
    small = _last(z, 5)
    ps, js = E.topk_routing_fwd(small, k)
    assert torch.equal(p[-5:], ps) and torch.equal(i[-5:], js)
    dz = E.topk_routing_bwd(p, z, i)
    assert torch.equal(dz[-5:], E.topk_routing_bwd(ps, small, js))


def _codes(rows, K, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    q = torch.randint(0, 256, (rows, K // 2), dtype=torch.uint8, device=DEV, generator=g)
    return q, torch.randint(125, 129, (rows, K // 32), dtype=torch.uint8, device=DEV, generator=g)


def test_offsets_past_32_bits_products():
    """One block of 32 sums exactly in every kernel: the last outputs are those of a small call."""
    require_gpu()
    for M, N, tiles in ((70000, 32768, True), (64, 1 << 25, False)):
        note(f"4-bit product {M} x {N}")
        a, b = _codes(M, 32, 1), _codes(N, 32, 2)
        y = E.mxfp4_matmul(*a, *b)
        assert y.numel() >= 2 ** 31 and (E.mxfp4_matmul_workspace_size(M, N, 32) > 0) == tiles
        small = E.mxfp4_matmul(*(_last(t, 5) for t in a), *(_last(t, 200) for t in b))
        assert torch.equal(y[-5:, -200:], small)
        del y
    Ex, N, K = 40, 16384, 8192
    b = [t.view(Ex, N, -1) for t in _codes(Ex * N, K, 3)]
    assert b[0].numel() > 2 ** 31
    for M in (3, 2000):                                    # few rows, tiles
        note(f"4-bit product by expert, {M} rows, weights past 32 bits")
        a = _codes(M, K, 4)
        off = torch.zeros(Ex + 1, dtype=torch.int32, device=DEV)
        off[-1] = M
        y = E.mxfp4_grouped_matmul(*a, *b, off, out_dtype=F32)
        av, bv = (E.mxfp4_dequantize(*t, F32).double() for t in (tuple(u[-3:].contiguous() for u in a), tuple(u[-1] for u in b)))
        want, mag = (u[0].matmul(u[1]) for u in ((av, bv.t().contiguous()), (av.abs(), bv.abs().t().contiguous())))
        assert ((y[-3:].double() - want).abs() <= (K / 128 + 24) * 2.0 ** -22 * mag + 2.0 ** -24 * want.abs()).all()
