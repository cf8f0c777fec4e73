"""One workspace dict used by calls that run side by side on several streams,
and by a captured graph beside eager calls: every result has to be that of the
call alone, bit for bit."""
import pytest
import torch

import group_sparse_swiglu_amd as E
from gpu_common import DEV, note, require_gpu

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _layer(T, Ex, d, ff, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, d, generator=g).to(BF)
    r = (torch.randn(Ex, d, generator=g) * d ** -0.5).to(BF)
    ws = [(torch.randn(Ex, *s, generator=g) * s[1] ** -0.5).to(BF) for s in ((ff, d), (ff, d), (d, ff))]
    return [t.to(DEV) for t in (x, r, 0.1 * torch.rand(Ex, generator=g), *ws)]


def test_overlapping_streams_share_a_dict():
    require_gpu()
    note("streams share a dict")
    layers = [_layer(T, 48, 512, 272, T) for T in (1, 7, 40)]
    want = [E.moe_decode(*a, 6) for a in layers]
    g = torch.Generator().manual_seed(5)
    pairs = [[E.fp8_quantize(torch.randn(128, 8208, generator=g).to(BF).to(DEV)) for _ in range(2)] for _ in layers]
    wanty = [E.fp8_matmul(*p, *q) for p, q in pairs]
    cache, outs = {}, []
    streams = [torch.cuda.Stream() for _ in layers]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                (a, b), layer = pairs[i], layers[i]
                outs.append((i, E.moe_decode(*layer, 6, workspace=cache), E.fp8_matmul(*a, *b, workspace=cache)))
    torch.cuda.synchronize()
    for i, got, y in outs:
        assert all(torch.equal(u, v) for u, v in zip(got, want[i])) and torch.equal(y, wanty[i])


def test_a_graph_keeps_its_scratch_while_the_dict_grows():
    require_gpu()
    note("graph beside a growing dict")
    small, large = _layer(3, 48, 512, 272, 1), _layer(64, 48, 512, 272, 2)
    want, wantl = E.moe_decode(*small, 6), E.moe_decode(*large, 6)
    cache = {}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        E.moe_decode(*small, 6, workspace=cache)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = E.moe_decode(*small, 6, workspace=cache)
    for _ in range(3):
        for t in out:
            t.zero_()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):               # beside the replay, on the stream of the capture
            got = E.moe_decode(*large, 6, workspace=cache)
            junk = [torch.full((1 << 18,), 7, dtype=torch.int32, device=DEV) for _ in range(4)]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(out, want))
        assert all(torch.equal(u, v) for u, v in zip(got, wantl))
        del junk
