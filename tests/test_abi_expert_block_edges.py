"""Edges of the norm, the routing with groups and the 4-bit operators that need no GPU."""
import ctypes

import pytest
import torch

import group_sparse_swiglu_amd as E

P = 64  # an aligned, never dereferenced address
NULL = None


def _caller(f, names, ok):
    return lambda **kw: f(*[kw.get(n, v) for n, v in zip(names, ok)])


def test_products_by_expert_of_no_rows():
    """Without rows in a nothing of it is read, and an empty tensor's address is NULL."""
    names = ("a", "sa", "R", "rows", "b", "sb", "E", "off", "dt", "M", "N", "K", "y", "ws", "bytes", "stream")
    call = _caller(E.lib().esg_mxfp4_grouped_matmul, names, (P, P, 9, P, P, P, 3, P, 1, 12288, 4096, 64, P, NULL, 0, NULL))
    assert call() == 3                                     # all is well but the workspace
    assert call(R=0, a=NULL, sa=NULL) == 3 and call(R=0) == 3
    assert call(a=NULL) == 1 and call(sa=NULL) == 1
    assert call(R=0, rows=NULL) == 1 and call(R=0, a=P + 8) == 1


@pytest.fixture
def launches(monkeypatch):
    """The autograd paths on CPU tensors, the launches stood in for: name -> arguments, and what lay at the inputs' addresses."""
    seen, real, dev = [], E.lib(), E._dev

    class Lib:
        def __getattr__(self, name):
            if name.endswith(("_size", "_string")):
                return getattr(real, name)

            def launch(*args):
                if name == "esg_rms_norm_bwd":
                    dy, dh, h, w, rstd, code, w_code, T, d = args[:9]
                    read = {k: ctypes.string_at(p, n * (4 if c == 0 else 2)) for k, p, n, c in
                            (("dy", dy, T * d, code), ("h", h, T * d, code), ("weight", w, d, w_code))}
                    seen.append({**read, "code": code, "rstd": ctypes.string_at(rstd, 4 * T)})
                if name == "esg_topk_routing_bwd":
                    dp, z, code, idx, T, n, k = args[:7]
                    seen.append(dict(dprobs=ctypes.string_at(dp, 4 * T * k), indices=ctypes.string_at(idx, 4 * T * k),
                                     logits=ctypes.string_at(z, T * n * (4 if code == 0 else 2)), code=code))
                return 0

            return launch

    monkeypatch.setattr(E, "lib", Lib)
    monkeypatch.setattr(E, "_stream", lambda dev: 0)
    monkeypatch.setattr(E, "_dev", lambda t, name, dtype=None, on=None: None if t is None else dev(
        t, name, dtype, t.get_device() if on is None else on))
    return seen


def _bytes(t):
    return t.detach().contiguous().view(torch.uint8).numpy().tobytes()


def _strided(t):
    """t's values, every other element of a larger buffer."""
    return torch.stack((t, t), -1)[..., 0] if t.dim() else t


def _through(hook):
    return torch.autograd.graph.saved_tensors_hooks(lambda t: t.detach().clone(), hook)


def test_saved_tensors_may_come_back_strided(launches):
    x, w = torch.randn(5, 64).bfloat16().requires_grad_(), torch.randn(64, requires_grad=True)
    with _through(_strided):
        y = E.rms_norm(x, w)
    torch.autograd.grad(y, (x, w), torch.ones_like(y))
    assert launches[-1]["h"] == _bytes(x) and launches[-1]["weight"] == _bytes(w)
    z = torch.randn(5, 16).bfloat16().requires_grad_()
    with _through(_strided):
        p, idx = E.topk_routing(z, 2)
        kept = idx.clone()
    torch.autograd.grad(p, z, torch.ones_like(p))
    assert launches[-1]["logits"] == _bytes(z) and launches[-1]["indices"] == _bytes(kept)


def test_saved_tensors_of_another_kind_are_refused(launches):
    for widen in (lambda t: t.float() if t.dtype == torch.bfloat16 else t, lambda t: t[:, :-16] if t.dim() == 2 else t):
        x, w = torch.randn(5, 64).bfloat16().requires_grad_(), torch.randn(64, requires_grad=True)
        with _through(widen):
            y = E.rms_norm(x, w)
        with pytest.raises(E.EsgError, match="h of the backward"):
            torch.autograd.grad(y, (x, w), torch.ones_like(y))
        z = torch.randn(5, 32).bfloat16().requires_grad_()
        with _through(lambda t: widen(t) if t.dtype == torch.bfloat16 else t):
            p, _ = E.topk_routing(z, 2)
        with pytest.raises(E.EsgError, match="logits of the backward"):
            torch.autograd.grad(p, z, torch.ones_like(p))
    assert not launches
    for bad in (dict(dtype=torch.float32), dict(gpu=1), dict(numel=7)):
        with pytest.raises(E.EsgError, match="here of the backward"):
            E._kept(torch.zeros(8).bfloat16(), **{**dict(dtype=torch.bfloat16, gpu=-1, numel=8, name="here"), **bad})


def test_tangents_are_not_dropped(launches):
    """The operators have no forward-mode gradient: a dual tensor is refused, whatever asks for reverse ones."""
    x, w, z = torch.randn(5, 64), torch.randn(64), torch.randn(5, 16)
    calls = {"x": lambda t: E.rms_norm(t, w), "w": lambda t: E.rms_norm(x, t), "r": lambda t: E.rms_norm(x, w, t),
             "z": lambda t: E.topk_routing(t, 2), "l": lambda t: E.fp8_linear(t, torch.randn(32, 64))}
    arg = {"x": x, "w": w, "r": x, "z": z, "l": x}
    for grad in (False, True):
        with torch.set_grad_enabled(grad), torch.autograd.forward_ad.dual_level():
            for name, call in calls.items():
                with pytest.raises(NotImplementedError, match="jvp"):
                    call(torch.autograd.forward_ad.make_dual(arg[name], torch.ones_like(arg[name])))
                call(arg[name])                            # without a tangent as ever


def test_norm_leaves_both_results():
    """y in the place of x and the new residual too would leave one of them."""
    names = ("x", "res", "w", "dt", "wdt", "T", "d", "eps", "y", "h", "rstd", "stream")
    call = _caller(E.lib().esg_rms_norm_fwd, names, (P, 2 * P, P, 1, 0, 4, 64, 1e-6, P, P, P, NULL))
    assert call() == 1 and call(y=3 * P, h=3 * P) == 1 and call(T=0) == 0
    names = ("x", "res", "w", "dt", "wdt", "T", "d", "eps", "qt", "q", "scale", "h", "stream")
    call = _caller(E.lib().esg_rms_norm_quant, names, (P, 2 * P, P, 1, 1, 4, 64, 1e-6, 2, 3 * P, P, 3 * P, NULL))
    assert call() == 1


def test_widths_and_counts_past_32_bits():
    """2^32 + 64 is not 64, whichever size it is.  (The message is that of too many rows; no tensor holds memory.)"""
    meta, n = dict(device="meta"), (1 << 32) + 64
    u8 = lambda *s: torch.empty(*s, dtype=torch.uint8, **meta)  # noqa: E731
    i32 = lambda *s: torch.empty(*s, dtype=torch.int32, **meta)  # noqa: E731
    x = torch.empty(2, n, **meta)
    z, p = torch.empty(0, 8, **meta), torch.empty(0, 2, **meta)
    calls = [lambda: E.rms_norm(x, x[0]), lambda: E.rms_norm_quantize(x, x[0]), lambda: E.mxfp4_quantize(x),
             lambda: E.mxfp4_dequantize(u8(2, n // 2), u8(2, n // 32)),
             lambda: E.mxfp4_matmul(u8(2, n // 2), u8(2, n // 32), u8(3, n // 2), u8(3, n // 32)),
             lambda: E.mxfp4_grouped_matmul(u8(2, n // 2), u8(2, n // 32), u8(1, 3, n // 2), u8(1, 3, n // 32), i32(2)),
             lambda: E.mxfp4_grouped_matmul(u8(2, 16), u8(2, 1), u8(n, 0, 16), u8(n, 0, 1), i32(n + 1)),
             lambda: E.topk_routing(z, n), lambda: E.topk_routing(z, 2, groups=n), lambda: E.topk_routing(z, 2, groups=4, topk_groups=n),
             lambda: E.topk_routing_bwd(p.expand(0, 2), torch.empty(0, n, **meta), i32(0, 2)),
             lambda: E.topk_routing_bwd(torch.empty(0, n, **meta), z, i32(0, n)),
             lambda: E.rms_norm_bwd_workspace_size(4, n), lambda: E.mxfp4_matmul_workspace_size(4, n, 64),
             lambda: E.mxfp4_matmul_workspace_size(4, 64, n), lambda: E.mxfp4_grouped_matmul_workspace_size(4, 4, 64, n),
             lambda: E.rms_norm_bwd_workspace_size(-n, 64)]
    for i, call in enumerate(calls):
        with pytest.raises(E.EsgError, match="rows, widths and counts"):
            print("call", i)
            call()
    ok = E.topk_routing_supported
    assert ok(64, 8) and not ok(n, 8) and not ok(64, (1 << 32) + 8) and not ok(64, 8, (1 << 32) + 1, 1) and not ok(64 - (1 << 32), 8)


def test_bias_strides_past_32_bits(launches):
    """The library takes the bias's stride in 32 bits."""
    bias = torch.zeros(1).as_strided((1,), (1,)).expand(8)
    far = type("Far", (), dict(dim=lambda s: 1, shape=torch.Size([8]), dtype=torch.float32, is_cuda=True, get_device=lambda s: -1,
                               stride=lambda s, i: (1 << 32) + 1))()
    with pytest.raises(E.EsgError, match="rows, widths and counts"):
        E.topk_routing_fwd(torch.zeros(4, 8), 2, expert_bias=far)
    with pytest.raises(E.EsgError, match="GPU"):
        E.topk_routing_fwd(torch.zeros(4, 8), 2, expert_bias=bias)
