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
    call = _caller(E.lib().esg_rms_norm_bwd, names, (P, NULL, P, P, P, 1, 1, 4, 64, P, P, P, 1 << 40, NULL))
    assert call(T=0, dw=NULL) == 0 and call(T=0, dw=NULL, dy=NULL, h=NULL) == 0
    for n in ("dy", "h", "w", "rstd", "dx"):
        assert call(**{n: NULL}) == 1
    for n in ("dy", "dh", "h", "w", "dx", "dw", "ws"):
        assert call(**{n: P + 8}) == 1
    assert call(ws=NULL) == 3 and call(bytes=0) == 3 and call(d=40) == 2 and call(T=-2) == 1
    assert E.rms_norm_bwd_workspace_size(0, 64) == 0
    assert E.rms_norm_bwd_workspace_size(5, 2048) >= 2048 * 4
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
