"""Argument checks of the 8-bit operators and of the expert layer for a few
tokens: every refusal returns before any launch.  CPU only."""
import ctypes

import pytest
import torch

import group_sparse_swiglu_amd as E

P = 64  # an aligned, never dereferenced address
NULL = None


def test_quant_rows_refusals():
    f = E.lib().esg_fp8_quant_rows
    assert f(P, 1, 0, 128, P, P, NULL, NULL, NULL) == 0            # no rows: nothing to do
    assert f(NULL, 1, 0, 128, NULL, NULL, NULL, NULL, NULL) == 0
    assert f(P, 2, 4, 128, P, P, NULL, NULL, NULL) == 2            # dtype
    assert f(P, 1, 4, 120, P, P, NULL, NULL, NULL) == 2            # cols % 16
    assert f(P, 1, 4, 0, P, P, NULL, NULL, NULL) == 1
    assert f(P, 1, -1, 128, P, P, NULL, NULL, NULL) == 1
    assert f(P, 1, 4, (1 << 22) + 16, P, P, NULL, NULL, NULL) == 2
    assert f(NULL, 1, 4, 128, P, P, NULL, NULL, NULL) == 1
    assert f(P, 1, 4, 128, NULL, P, NULL, NULL, NULL) == 1
    assert f(P, 1, 4, 128, P, NULL, NULL, NULL, NULL) == 1
    assert f(P + 8, 1, 4, 128, P, P, NULL, NULL, NULL) == 1        # misaligned
    assert f(P, 1, 4, 128, P + 8, P, NULL, NULL, NULL) == 1
    assert f(P, 1, 4, 128, P, P + 2, NULL, NULL, NULL) == 1
    assert f(P, 1, 4, 128, P, P, P, NULL, NULL) == 1               # qt without its scales
    assert f(P, 1, 4, 128, P, P, NULL, P, NULL) == 1
    assert f(P, 1, 4, 128, P, P, P + 4, P, NULL) == 1


def test_quant_tiles_refusals():
    f = E.lib().esg_fp8_quant_tiles
    assert f(P, 0, 0, 5, 128, P, P, NULL, NULL, NULL) == 0
    assert f(P, 0, 3, 0, 128, P, P, NULL, NULL, NULL) == 0
    assert f(P, 0, -1, 5, 128, P, P, NULL, NULL, NULL) == 1
    assert f(P, 0, 2, 5, 24, P, P, NULL, NULL, NULL) == 2
    assert f(P, 0, 1 << 20, 1 << 20, 1 << 20, P, P, NULL, NULL, NULL) == 2   # 2^31 tiles and more
    assert f(NULL, 0, 2, 5, 128, P, P, NULL, NULL, NULL) == 1
    assert f(P, 0, 2, 5, 128, P, P, P, NULL, NULL) == 1
    assert f(P, 7, 2, 5, 128, P, P, NULL, NULL, NULL) == 2


def _ws(M, N, K):
    need = ctypes.c_size_t()
    st = E.lib().esg_fp8_matmul_workspace_size(M, N, K, ctypes.byref(need))
    return st, need.value


def test_matmul_refusals_and_workspace():
    f = E.lib().esg_fp8_matmul
    ok = (P, P, P, P, 0, 1, 4, 32, 128, P, P, 1 << 40, NULL)

    def call(**kw):
        names = ("a", "sa", "b", "sb", "rows", "out", "M", "N", "K", "y", "ws", "bytes", "stream")
        return f(*[kw.get(n, v) for n, v in zip(names, ok)])

    assert call(M=0) == 0 and call(N=0) == 0 and call(M=0, a=NULL) == 0
    for name in ("a", "sa", "b", "sb", "y"):
        assert call(**{name: NULL}) == 1
    for name in ("a", "b", "y"):
        assert call(**{name: P + 8}) == 1
    for name in ("sa", "sb"):
        assert call(**{name: P + 2}) == 1
    assert call(M=-1) == 1 and call(K=0) == 1 and call(N=-3) == 1
    assert call(K=100) == 2 and call(K=(1 << 22) + 16) == 2 and call(out=2) == 2
    assert call(M=1 << 30, N=1 << 24) == 2 and call(N=(1 << 25) + 1) == 2   # more threads than a launch may have
    assert E.lib().esg_fp8_matmul_workspace_size(4, 4, 128, None) == 1
    assert _ws(4, 4, 100)[0] == 2
    assert _ws(4, 4096, 2048) == (0, 0)
    assert _ws(0, 128, 128) == (0, 0)
    # few output tiles and a long K: the K parts are added in the workspace
    st, need = _ws(128, 128, 16384)
    assert st == 0 and need >= 2 * 128 * 128 * 4
    assert call(M=128, N=128, K=16384, bytes=need - 1) == 3
    assert call(M=128, N=128, K=16384, ws=NULL) == 3
    assert call(M=128, N=128, K=16384, ws=P + 8) == 1


def test_linear_refusals_and_sizes():
    lib = E.lib()

    def sizes(*args):
        out = [ctypes.c_size_t() for _ in range(3)]
        return lib.esg_fp8_linear_workspace_size(*args, *map(ctypes.byref, out)), *(o.value for o in out)

    st, sv, fw, bw = sizes(100, 256, 512, 1, 1)
    assert st == 0 and sv >= 256 * 112 + 256 * 512 and fw >= 100 * 256 + 512 * 256 and bw >= 100 * 512 + 512 * 112
    assert sizes(100, 256, 512, 0, 0)[1] == 0
    assert sizes(100, 256, 512, 1, 0)[1] < sv and sizes(100, 256, 512, 0, 1)[1] < sv
    assert sizes(0, 256, 512, 1, 1)[0] == 0
    assert sizes(4, 250, 512, 1, 1)[0] == 2 and sizes(4, 256, 500, 1, 1)[0] == 2
    assert sizes(-1, 256, 512, 1, 1)[0] == 1 and sizes(4, 0, 512, 1, 1)[0] == 1
    assert lib.esg_fp8_linear_workspace_size(4, 256, 512, 1, 1, None, None, None) == 1
    f, big = lib.esg_fp8_linear_fwd, 1 << 40
    assert f(NULL, 1, P, 1, 4, 256, 512, 1, 1, P, P, big, P, big, NULL) == 1
    assert f(P, 1, NULL, 1, 4, 256, 512, 1, 1, P, P, big, P, big, NULL) == 1
    assert f(P, 1, P, 1, 4, 256, 512, 1, 1, P + 8, P, big, P, big, NULL) == 1
    assert f(P, 2, P, 1, 4, 256, 512, 1, 1, P, P, big, P, big, NULL) == 2
    assert f(P, 1, P, 2, 4, 256, 512, 1, 1, P, P, big, P, big, NULL) == 2
    assert f(P, 1, P, 1, 4, 256, 512, 1, 1, P, NULL, 0, P, big, NULL) == 3
    assert f(P, 1, P, 1, 4, 256, 512, 1, 1, P, P, 16, P, big, NULL) == 3
    assert f(P, 1, P, 1, 4, 256, 512, 1, 1, P, P, big, P, 16, NULL) == 3
    assert f(P, 1, P, 1, 4, 256, 512, 1, 1, P, P + 8, big, P, big, NULL) == 1
    b = lib.esg_fp8_linear_bwd
    assert b(P, 1, 1, 4, 256, 512, P, big, NULL, NULL, P, big, NULL) == 0        # nothing asked for
    assert b(NULL, 1, 1, 4, 256, 512, P, big, P, P, P, big, NULL) == 1
    assert b(P, 1, 1, 4, 256, 512, P, 16, P, P, P, big, NULL) == 3
    assert b(P, 1, 1, 4, 256, 512, P, big, P, P, P, 16, NULL) == 3
    assert b(P, 1, 1, 4, 256, 512, P, big, P + 8, P, P, big, NULL) == 1
    assert b(P, 3, 1, 4, 256, 512, P, big, P, P, P, big, NULL) == 2


def test_moe_refusals_and_workspace():
    lib = E.lib()
    sup = lib.esg_moe_decode_supported
    assert sup(1, 256, 8, 2048, 1024, 1) == 1 and sup(64, 1024, 32, 16, 16, 2) == 1 and sup(0, 1, 1, 16, 16, 1) == 1
    for bad in ((65, 8, 2, 64, 64, 1), (-1, 8, 2, 64, 64, 1), (1, 1025, 2, 64, 64, 1), (1, 8, 9, 64, 64, 1),
                (1, 64, 33, 64, 64, 1), (1, 8, 0, 64, 64, 1), (1, 8, 2, 72, 64, 1), (1, 8, 2, 64, 72, 1),
                (1, 8, 2, 64, 64, 0), (1, 8, 2, 64, 64, 3), (1, 8, 2, 0, 64, 1), (1, 8, 2, 64, 0, 1)):
        assert sup(*bad) == 0, bad
    need = ctypes.c_size_t()
    assert lib.esg_moe_decode_workspace_size(4, 8, 2, 64, 64, ctypes.byref(need)) == 0 and need.value > 0
    assert lib.esg_moe_decode_workspace_size(65, 8, 2, 64, 64, ctypes.byref(need)) == 2
    assert lib.esg_moe_decode_workspace_size(4, 8, 2, 64, 64, None) == 1
    names = ("x", "r", "b", "stride", "g", "u", "d", "sg", "su", "sd", "dt", "T", "E", "k", "dm", "ff", "f", "sc", "y",
             "p", "i", "ws", "bytes", "stream")
    ok = (P, P, P, 1, P, P, P, NULL, NULL, NULL, 1, 4, 8, 2, 64, 64, 1.0, 0, P, P, P, P, 1 << 30, NULL)

    def call(**kw):
        return lib.esg_moe_decode(*[kw.get(n, v) for n, v in zip(names, ok)])

    assert call(T=0) == 0 and call(T=0, x=NULL, ws=NULL) == 0
    for name in ("x", "r", "b", "g", "u", "d", "y", "p", "i"):
        assert call(**{name: NULL}) == 1
    for name in ("x", "r", "g", "u", "d", "y", "ws"):
        assert call(**{name: P + 8}) == 1
    assert call(stride=0) == 1 and call(T=-1) == 1 and call(T=65) == 2 and call(dt=0) == 2
    assert call(dt=2) == 1                                         # 8-bit weights without scales
    assert call(ws=NULL) == 3 and call(bytes=16) == 3


def test_python_checks_raise_without_a_gpu():
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    with pytest.raises(E.EsgError):
        E.fp8_quantize(x)                                          # not a GPU tensor
    with pytest.raises(E.EsgError):
        E.fp8_quantize(x[0])
    with pytest.raises(E.EsgError):
        E.fp8_quantize(x.half())
    with pytest.raises(E.EsgError):
        E.fp8_quantize_weight(x.view(1, 1, 4, 128))
    q, s = torch.zeros(4, 128, dtype=torch.float8_e4m3fn), torch.zeros(4, 1)
    with pytest.raises(E.EsgError):
        E.fp8_matmul(q, s, q[:, :64], s)
    with pytest.raises(E.EsgError):
        E.fp8_matmul(q, s[:3], q, s)
    with pytest.raises(E.EsgError):
        E.fp8_matmul(q, s, q, s[:2])
    with pytest.raises(E.EsgError):
        E.fp8_linear(x, torch.zeros(24, 128))
    with pytest.raises(E.EsgError):
        E.fp8_linear(x, torch.zeros(32, 64))
    w = torch.zeros(8, 32, 128, dtype=torch.bfloat16)
    r, b = torch.zeros(8, 128, dtype=torch.bfloat16), torch.zeros(8)
    with pytest.raises(E.EsgError):
        E.moe_decode(x, r, b, w, w, w, 2)                          # w_down must be [E, d, ff]
    with pytest.raises(E.EsgError):
        E.moe_decode(x, r, b, w.half(), w.half(), w.half().transpose(1, 2).contiguous(), 2)
    w8 = w.to(torch.float8_e4m3fn)
    with pytest.raises(E.EsgError):
        E.moe_decode(x, r, b, w8, w8, w8.transpose(1, 2).contiguous(), 2)   # no scales
    with pytest.raises(E.EsgError):
        E.moe_decode(x, r, b[:7], w, w, w.transpose(1, 2).contiguous(), 2)
    assert E.moe_decode_supported(64, 256, 8, 2048, 1024)
    assert E.moe_decode_supported(64, 256, 8, 2048, 1024, torch.float8_e4m3fn)
    assert not E.moe_decode_supported(64, 256, 8, 2048, 1024, torch.float32)
