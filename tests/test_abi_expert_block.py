"""Argument checks of the norm, the routing with groups and the 4-bit operators:
every refusal returns before any launch.  CPU only."""
import ctypes

import pytest
import torch

import group_sparse_swiglu_amd as E

P = 64  # an aligned, never dereferenced address
NULL = None


def _caller(f, names, ok):
    return lambda **kw: f(*[kw.get(n, v) for n, v in zip(names, ok)])


def test_norm_refusals():
    names = ("x", "res", "w", "dt", "wdt", "T", "d", "eps", "y", "h", "rstd", "stream")
    call = _caller(E.lib().esg_rms_norm_fwd, names, (P, P, P, 1, 0, 4, 64, 1e-6, P, P, P, NULL))
    assert call(T=0) == 0 and call(T=0, x=NULL) == 0
    assert call(T=-1) == 1 and call(d=0) == 1
    assert call(dt=2) == 2 and call(wdt=3) == 2 and call(d=24) == 2 and call(d=16400) == 2
    for n in ("x", "w", "y"):
        assert call(**{n: NULL}) == 1
    for n in ("x", "res", "w", "y", "h"):
        assert call(**{n: P + 8}) == 1
    assert call(res=NULL) == 1 and call(h=NULL) == 1 and call(rstd=P + 2) == 1


def test_norm_quant_refusals():
    names = ("x", "res", "w", "dt", "wdt", "T", "d", "eps", "qt", "q", "scale", "h", "stream")
    call = _caller(E.lib().esg_rms_norm_quant, names, (P, NULL, P, 1, 1, 4, 64, 1e-6, 2, P, P, NULL, NULL))
    assert call(T=0) == 0
    assert call(qt=1) == 2 and call(qt=4) == 2 and call(qt=3, d=48) == 2 and call(d=24) == 2
    assert call(scale=NULL) == 1 and call(scale=P + 2) == 1 and call(q=P + 4) == 1 and call(h=P) == 1


def test_norm_backward_refusals_and_workspace():
    names = ("dy", "dh", "h", "w", "rstd", "dt", "wdt", "T", "d", "dx", "dw", "ws", "bytes", "stream")
    call = _caller(E.lib().esg_rms_norm_bwd, names, (P, NULL, P, P, P, 1, 1, 4, 64, 2 * P, P, P, 1 << 40, NULL))
    assert call(dx=P) == 1                                  # dy itself, which dw still needs
    assert call(T=0, dw=NULL) == 0 and call(T=0, dw=NULL, dy=NULL, h=NULL) == 0
    for n in ("dy", "h", "w", "rstd", "dx"):
        assert call(**{n: NULL}) == 1
    for n in ("dy", "dh", "h", "w", "dx", "dw", "ws"):
        assert call(**{n: P + 8}) == 1
    assert E.rms_norm_bwd_workspace_size(5000, 64) > 0
    assert call(T=5000, ws=NULL) == 3 and call(T=5000, bytes=0) == 3 and call(d=40) == 2 and call(T=-2) == 1
    assert E.rms_norm_bwd_workspace_size(0, 64) == 0
    assert E.rms_norm_bwd_workspace_size(5, 2048) == 0 and E.rms_norm_bwd_workspace_size(5000, 2048) >= 2048 * 4
    assert E.rms_norm_bwd_workspace_size(1 << 30, 16384) <= 1 << 27
    need = ctypes.c_size_t()
    assert E.lib().esg_rms_norm_bwd_workspace_size(4, 50, ctypes.byref(need)) == 2
    assert E.lib().esg_rms_norm_bwd_workspace_size(4, 64, NULL) == 1


def test_routing_refusals():
    names = ("z", "dt", "bias", "bs", "T", "E", "k", "score", "G", "kg", "norm", "c", "p", "i", "stream")
    call = _caller(E.lib().esg_topk_routing_fwd, names, (P, 0, P, 1, 4, 64, 8, 0, 8, 4, 1, 1.0, P, P, NULL))
    assert call(T=0) == 0 and call(T=0, z=NULL) == 0
    assert call(T=-1) == 1 and call(bs=0) == 1
    for n in ("z", "p", "i"):
        assert call(**{n: NULL}) == 1 and call(**{n: P + 1}) == 1
    assert call(bias=P + 2) == 1
    assert call(dt=2) == 2 and call(score=2) == 2 and call(k=0) == 2 and call(k=33) == 2
    assert call(kg=1, k=9) == 2 and call(G=7) == 2 and call(kg=9) == 2 and call(kg=0) == 2
    assert call(T=1 << 26) == 2
    names = ("dp", "z", "dt", "i", "T", "E", "k", "score", "norm", "c", "dz", "stream")
    call = _caller(E.lib().esg_topk_routing_bwd, names, (P, P, 1, P, 4, 64, 8, 1, 1, 1.0, P, NULL))
    assert call(T=0) == 0
    for n in ("dp", "z", "i", "dz"):
        assert call(**{n: NULL}) == 1 and call(**{n: P + 1}) == 1
    assert call(E=4) == 2 and call(dt=3) == 2 and call(E=1025) == 2


def test_routing_shapes():
    ok = E.topk_routing_supported
    assert ok(1, 1) and ok(1024, 32) and ok(256, 8, 8, 4) and ok(384, 12, 6, 2) and ok(64, 1, 64, 1) and not ok(64, 2, 64, 1) and ok(2, 1, 2, 1)
    assert not ok(1025, 1) and not ok(1024, 33) and not ok(8, 9) and not ok(130, 1, 65, 1) and not ok(10, 1, 3, 1)
    assert ok(130, 1, 65, 65)                                   # every group stays: they do not matter
    assert ok(16 * 64, 4, 8, 2) and not ok(17 * 48, 4, 48, 2) and ok(16 * 48, 4, 48, 2)


def test_four_bit_refusals():
    q, d = E.lib().esg_mxfp4_quant, E.lib().esg_mxfp4_dequant
    assert q(P, 1, 0, 32, P, P, NULL) == 0 and d(P, P, 1, 0, 32, P, NULL) == 0
    assert q(P, 2, 4, 32, P, P, NULL) == 2 and q(P, 1, 4, 48, P, P, NULL) == 2 and q(P, 1, 4, 0, P, P, NULL) == 1
    assert q(P, 1, -1, 32, P, P, NULL) == 1 and q(P, 1, 4, (1 << 22) + 32, P, P, NULL) == 2
    assert q(P, 1, 1 << 40, 64, P, P, NULL) == 2
    assert q(NULL, 1, 4, 32, P, P, NULL) == 1 and q(P, 1, 4, 32, NULL, P, NULL) == 1 and q(P, 1, 4, 32, P, NULL, NULL) == 1
    assert q(P + 8, 1, 4, 32, P, P, NULL) == 1 and q(P, 1, 4, 32, P + 8, P, NULL) == 1
    assert d(P, P, 3, 4, 32, P, NULL) == 2 and d(P, NULL, 1, 4, 32, P, NULL) == 1 and d(P, P, 1, 4, 32, P + 4, NULL) == 1


def test_binding_refusals():
    x, w = torch.zeros(4, 64), torch.zeros(64)
    with pytest.raises(E.EsgError, match="weight"):
        E.rms_norm(x, torch.zeros(32))
    with pytest.raises(E.EsgError, match="residual must have"):
        E.rms_norm(x, w, x.bfloat16())
    with pytest.raises(E.EsgError, match="residual must have"):
        E.rms_norm_quantize(x, w, torch.zeros(3, 64))
    with pytest.raises(E.EsgError, match="format"):
        E.rms_norm_quantize(x, w, format="int8")
    with pytest.raises(E.EsgError, match="residual_out"):
        E.rms_norm_quantize(x, w, residual_out=x)
    with pytest.raises(E.EsgError, match="GPU tensor"):
        E.rms_norm_fwd(x, w)
    with pytest.raises(E.EsgError, match="scoring"):
        E.topk_routing(torch.zeros(4, 8), 2, "linear")
    with pytest.raises(E.EsgError, match="num_experts"):
        E.topk_routing(torch.zeros(8), 2)
    with pytest.raises(E.EsgError, match="expert_bias"):
        E.topk_routing(torch.zeros(4, 8), 2, expert_bias=torch.zeros(7))
    with pytest.raises(E.EsgError, match="indices"):
        E.topk_routing_bwd(torch.zeros(4, 2), torch.zeros(4, 8), torch.zeros(4, 3, dtype=torch.int32))
    with pytest.raises(E.EsgError, match="scale"):
        E.mxfp4_dequantize(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 1, dtype=torch.uint8))
    with pytest.raises(E.EsgError, match="GPU tensor"):
        E.mxfp4_quantize(x)


def test_four_bit_product_refusals():
    names = ("a", "sa", "b", "sb", "dt", "M", "N", "K", "y", "ws", "bytes", "stream")
    call = _caller(E.lib().esg_mxfp4_matmul, names, (P, P, P, P, 1, 4, 16, 64, P, NULL, 0, NULL))
    assert call(M=0) == 0 and call(N=0) == 0 and call(M=0, a=NULL, y=NULL) == 0 and call(M=0, dt=2) == 2
    assert call(M=-1) == 1 and call(N=-1) == 1 and call(K=0) == 1 and call(K=-32) == 1
    assert call(K=48) == 2 and call(K=(1 << 22) + 32) == 2 and call(dt=2) == 2 and call(dt=-1) == 2
    assert call(M=(1 << 30) + 1) == 2 and call(N=(1 << 25) + 1) == 2 and call(M=1 << 30, N=1 << 10) == 2
    for n in ("a", "b", "y"):
        assert call(**{n: NULL}) == 1 and call(**{n: P + 8}) == 1
    assert call(sa=NULL) == 1 and call(sb=NULL) == 1
    big = dict(M=4096, N=4096, K=2048)
    assert E.mxfp4_matmul_workspace_size(*big.values()) > 16
    assert call(**big) == 3 and call(**big, ws=P, bytes=16) == 3 and call(**big, ws=P + 8, bytes=1 << 40) == 1


def test_four_bit_product_by_expert_refusals():
    names = ("a", "sa", "R", "rows", "b", "sb", "E", "off", "dt", "M", "N", "K", "y", "ws", "bytes", "stream")
    call = _caller(E.lib().esg_mxfp4_grouped_matmul, names, (P, P, 9, P, P, P, 3, P, 1, 4, 16, 64, P, NULL, 0, NULL))
    assert call(M=0) == 0 and call(N=0) == 0 and call(M=0, dt=3) == 2
    assert call(M=-1) == 1 and call(K=0) == 1 and call(E=0) == 1 and call(R=-1) == 1
    assert call(rows=NULL, R=3) == 1                       # every row of y has one of a
    assert call(K=80) == 2 and call(E=1025) == 2 and call(dt=2) == 2
    assert call(K=64, R=(1 << 26)) == 2 and call(M=1 << 29, N=1 << 10) == 2    # rows are gathered at 32-bit offsets
    for n in ("a", "b", "y"):
        assert call(**{n: NULL}) == 1 and call(**{n: P + 8}) == 1
    for n in ("sa", "sb", "off"):
        assert call(**{n: NULL}) == 1
    assert call(rows=P + 2) == 1 and call(off=P + 2) == 1
    assert E.mxfp4_grouped_matmul_workspace_size(12288, 4096, 64, 3) > 100
    assert call(M=12288, N=4096) == 3 and call(M=12288, N=4096, ws=P, bytes=100) == 3


def test_four_bit_product_workspaces():
    for f, args in ((E.lib().esg_mxfp4_matmul_workspace_size, (64, 64, 64)),
                    (E.lib().esg_mxfp4_grouped_matmul_workspace_size, (64, 64, 64, 4))):
        need = ctypes.c_size_t(7)
        assert f(*args, NULL) == 1 and f(*args, ctypes.byref(need)) == 0 and need.value == 0
        assert f(-1, *args[1:], ctypes.byref(need)) == 1 and f(64, 64, 40, *args[3:], ctypes.byref(need)) == 2
    assert E.mxfp4_matmul_workspace_size(0, 64, 64) == 0 and E.mxfp4_matmul_workspace_size(1, 1 << 20, 64) == 0
    # one word for every 128 elements of a row of either side
    assert E.mxfp4_matmul_workspace_size(8192, 4096, 160) == (8192 + 4096) * 2 * 4
    assert E.mxfp4_grouped_matmul_workspace_size(12288, 4096, 160, 8) == (12288 + 8 * 4096) * 2 * 4
    with pytest.raises(E.EsgError):
        E.mxfp4_matmul_workspace_size(4, 4, 33)
    with pytest.raises(E.EsgError):
        E.mxfp4_grouped_matmul_workspace_size(4, 4, 32, 0)


def test_four_bit_product_binding_refusals():
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    a, sa, b, sb = u8(4, 32), u8(4, 2), u8(8, 32), u8(8, 2)
    for bad in ((u8(4, 16), sa, b, sb), (a[0], sa, b, sb), (a, sa, b[None], sb)):
        with pytest.raises(E.EsgError, match="K/2"):
            E.mxfp4_matmul(*bad)
    for bad in ((a, u8(4, 1), b, sb), (a, sa, b, u8(7, 2))):
        with pytest.raises(E.EsgError, match="K/32"):
            E.mxfp4_matmul(*bad)
    with pytest.raises(E.EsgError, match="out must be"):
        E.mxfp4_matmul(a, sa, b, sb, out=torch.zeros(4, 7))
    with pytest.raises(E.EsgError, match="dtype"):
        E.mxfp4_matmul(a, sa, b, sb, out_dtype=torch.float16)
    with pytest.raises(E.EsgError, match="GPU tensor"):
        E.mxfp4_matmul(a, sa, b, sb)
    b, sb, off = u8(3, 8, 32), u8(3, 8, 2), torch.zeros(4, dtype=torch.int32)
    for bad in ((a, sa, b[0], sb, off), (u8(4, 64), u8(4, 4), b, sb, off)):
        with pytest.raises(E.EsgError, match="K/2"):
            E.mxfp4_grouped_matmul(*bad)
    with pytest.raises(E.EsgError, match="K/32"):
        E.mxfp4_grouped_matmul(a, sa, b, u8(3, 8, 1), off)
    for kw in (dict(offsets=off[:3]), dict(offsets=off, rows=torch.zeros(2, 2, dtype=torch.int32))):
        with pytest.raises(E.EsgError, match="offsets"):
            E.mxfp4_grouped_matmul(a, sa, b, sb, **kw)
    with pytest.raises(E.EsgError, match="out must be"):
        E.mxfp4_grouped_matmul(a, sa, b, sb, off, rows=torch.zeros(9, dtype=torch.int32), out=torch.zeros(4, 8))
    with pytest.raises(E.EsgError, match="GPU tensor"):
        E.mxfp4_grouped_matmul(a, sa, b, sb, off)


def test_more_rows_than_the_library_counts():
    """2^32 + 1 rows are not one."""
    meta = dict(device="meta")
    n = (1 << 32) + 1
    with pytest.raises(E.EsgError, match="rows"):
        E.rms_norm(torch.empty(n, 16, **meta), torch.empty(16, **meta))
    with pytest.raises(E.EsgError, match="rows"):
        E.rms_norm_quantize(torch.empty(n, 16, **meta), torch.empty(16, **meta))
    with pytest.raises(E.EsgError, match="rows"):
        E.topk_routing(torch.empty(n, 4, **meta), 2)
    with pytest.raises(E.EsgError, match="rows"):
        E.topk_routing_bwd(torch.empty(n, 1, **meta), torch.empty(n, 4, **meta), torch.empty(n, 1, **meta))
    u8 = dict(dtype=torch.uint8, **meta)
    a, sa = torch.empty(n, 16, **u8), torch.empty(n, 1, **u8)
    b, sb = torch.empty(4, 16, **u8), torch.empty(4, 1, **u8)
    for args in ((a, sa, b, sb), (b, sb, a, sa)):
        with pytest.raises(E.EsgError, match="rows"):
            E.mxfp4_matmul(*args)
    with pytest.raises(E.EsgError, match="rows"):
        E.mxfp4_grouped_matmul(a, sa, b[None], sb[None], torch.empty(2, dtype=torch.int32, **meta))
