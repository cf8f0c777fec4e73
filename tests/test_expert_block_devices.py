"""The norm, the routing with groups and the 4-bit operators refuse tensors on different
GPUs before any launch.  CPU only: tensors and the library are stood in for."""
import pytest
import torch

import group_sparse_swiglu_amd as E
from test_fp8_moe_devices import HERE, OTHER, Stub, _each_elsewhere, launches  # noqa: F401

BF, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


@pytest.fixture(autouse=True)
def _likes(monkeypatch):
    monkeypatch.setattr(torch, "empty_like", lambda t, memory_format=None: Stub(t.shape, t.dtype, t.device))


def test_norm(launches):
    x = lambda: Stub((5, 64), BF)  # noqa: E731
    _each_elsewhere(lambda **kw: E.rms_norm_fwd(**kw),
                    dict(x=x(), weight=Stub((64,), F32), residual=x(), out=x(), residual_out=x()), launches)
    launches.clear()
    _each_elsewhere(lambda **kw: E.rms_norm_quantize(**kw),
                    dict(x=x(), weight=Stub((64,), F32), residual=x(), residual_out=x()), launches)
    launches.clear()
    _each_elsewhere(lambda **kw: E.rms_norm_bwd(**kw),
                    dict(dy=x(), h=x(), weight=Stub((64,), F32), rstd=Stub((5,), F32), dh=x()), launches)


def test_routing(launches):
    out = (Stub((5, 2), F32), Stub((5, 2), I32))
    _each_elsewhere(lambda **kw: E.topk_routing_fwd(topk=2, **kw),
                    dict(logits=Stub((5, 8), BF), expert_bias=Stub((8,), F32), out=out), launches)
    launches.clear()
    _each_elsewhere(lambda **kw: E.topk_routing_bwd(**kw),
                    dict(dprobs=Stub((5, 2), F32), logits=Stub((5, 8), BF), indices=Stub((5, 2), I32)), launches)


def test_four_bit(launches):
    _each_elsewhere(lambda **kw: E.mxfp4_dequantize(**kw), dict(q=Stub((4, 32), U8), scale=Stub((4, 2), U8)), launches)
    launches.clear()
    _each_elsewhere(lambda **kw: E.mxfp4_matmul(**kw),
                    dict(a=Stub((4, 32), U8), a_scale=Stub((4, 2), U8), b=Stub((8, 32), U8), b_scale=Stub((8, 2), U8),
                         out=Stub((4, 8), BF)), launches)
    launches.clear()
    _each_elsewhere(lambda **kw: E.mxfp4_grouped_matmul(**kw),
                    dict(a=Stub((4, 32), U8), a_scale=Stub((4, 2), U8), b=Stub((3, 8, 32), U8), b_scale=Stub((3, 8, 2), U8),
                         offsets=Stub((4,), I32), rows=Stub((6,), I32), out=Stub((6, 8), BF)), launches)


def test_the_wrong_types(launches):
    a, sa, b, sb = Stub((4, 32), U8), Stub((4, 2), U8), Stub((8, 32), U8), Stub((8, 2), U8)
    for args in ((Stub((4, 32), torch.int8), sa, b, sb), (a, Stub((4, 2), torch.int8), b, sb)):
        with pytest.raises(E.EsgError, match="uint8"):
            E.mxfp4_matmul(*args)
    with pytest.raises(E.EsgError, match="int32"):
        E.mxfp4_grouped_matmul(a, sa, Stub((1, 8, 32), U8), Stub((1, 8, 2), U8), Stub((2,), torch.int64))
    with pytest.raises(E.EsgError, match="float32"):
        E.rms_norm_bwd(Stub((5, 64), BF), Stub((5, 64), BF), Stub((64,), F32), Stub((5,), BF))
    with pytest.raises(E.EsgError, match="int32"):
        E.topk_routing_bwd(Stub((5, 2), F32), Stub((5, 8), BF), Stub((5, 2), torch.int64))
    assert not launches
    assert HERE != OTHER
