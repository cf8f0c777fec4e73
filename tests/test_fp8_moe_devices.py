"""Tensors on different GPUs are refused before any launch.  CPU only: tensors
and the library are stood in for."""
import pytest
import torch

import group_sparse_swiglu_amd as E

BF, F32, E4M3, I64 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.int64
HERE, OTHER = torch.device("cuda", 0), torch.device("cuda", 1)


class Stub:
    """As much of a contiguous GPU tensor as the calls look at."""

    is_cuda = True

    def __init__(self, shape, dtype, device=HERE):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, device

    def get_device(self):
        return self.device.index

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True

    def stride(self, i):
        return 1

    def data_ptr(self):
        return 4096


@pytest.fixture
def launches(monkeypatch):
    seen, real = [], E.lib()

    class Lib:
        def __getattr__(self, name):
            if name.endswith(("_size", "_string")):
                return getattr(real, name)
            return lambda *args: seen.append(name) or 0

    monkeypatch.setattr(E, "lib", Lib)
    monkeypatch.setattr(E, "_stream", lambda dev: 0)
    monkeypatch.setattr(E, "_ws", lambda n, dev, cache, key: Stub((max(n, 1),), torch.uint8, dev))
    monkeypatch.setattr(torch, "empty", lambda *s, dtype, device: Stub(s, dtype, device))
    return seen


def _each_elsewhere(call, args, launches):
    """call(**args) launches; with any one tensor (or one of a tuple) on the other GPU it is refused."""
    call(**args)
    assert len(launches) == 1
    for name, t in args.items():
        for i in range(len(t) if isinstance(t, tuple) else 1):
            moved = [Stub(u.shape, u.dtype, u.device) for u in (t if isinstance(t, tuple) else (t,))]
            moved[i].device = OTHER
            with pytest.raises(E.EsgError, match="cuda|GPU"):
                call(**{**args, name: tuple(moved) if isinstance(t, tuple) else moved[0]})
    assert len(launches) == 1


def test_matmul(launches):
    args = dict(a=Stub((40, 256), E4M3), a_scale=Stub((40, 2), F32), b=Stub((48, 256), E4M3),
                b_scale=Stub((1, 2), F32), out=Stub((40, 48), BF))
    call = lambda **kw: E.fp8_matmul(**kw)  # noqa: E731
    _each_elsewhere(call, args, launches)


def test_linear(launches):
    call = lambda x, w, out: E.fp8_linear_fwd(x, w, out=out)  # noqa: E731
    _each_elsewhere(call, dict(x=Stub((5, 128), BF), w=Stub((32, 128), F32), out=Stub((5, 32), BF)), launches)
    launches.clear()
    sv = E.fp8_linear_workspace_size(5, 128, 32)[0]
    call = lambda dy, saved: E.fp8_linear_bwd(dy, saved, 128, F32)  # noqa: E731
    _each_elsewhere(call, dict(dy=Stub((5, 32), BF), saved=Stub((sv,), torch.uint8)), launches)


def test_experts(launches):
    T, Ex, d, ff, k = 4, 8, 128, 64, 2
    args = dict(x=Stub((T, d), BF), w_router=Stub((Ex, d), BF), expert_bias=Stub((Ex,), F32),
                w_gate=Stub((Ex, ff, d), E4M3), w_up=Stub((Ex, ff, d), E4M3), w_down=Stub((Ex, d, ff), E4M3),
                scales=tuple(Stub((Ex, 1, 1), F32) for _ in range(3)),
                out=(Stub((T, d), BF), Stub((T, k), F32), Stub((T, k), I64)))
    _each_elsewhere(lambda **kw: E.moe_decode(topk=k, **kw), args, launches)


@pytest.mark.parametrize("n", [0, 2, 4])
def test_experts_take_three_scales(launches, n):
    w, wd = Stub((8, 64, 128), E4M3), Stub((8, 128, 64), E4M3)
    with pytest.raises(E.EsgError, match="three"):
        E.moe_decode(Stub((4, 128), BF), Stub((8, 128), BF), Stub((8,), F32), w, w, wd, 2,
                     scales=tuple(Stub((8, 1, 1), F32) for _ in range(n)))
    assert not launches
