"""Scratch buffers in a caller's dict: none is shared by calls that may run side
by side or by a captured graph.  CPU only: streams, capture and allocation are
stood in for."""
import pytest
import torch

import group_sparse_swiglu_amd as E

DEV = torch.device("cuda", 0)


@pytest.fixture
def device(monkeypatch):
    state = dict(stream=11, capturing=False)

    class Buffer:
        device = DEV

        def __init__(self, n):
            self.n = n

        def numel(self):
            return self.n

    monkeypatch.setattr(E, "_stream", lambda dev: state["stream"])
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state["capturing"])
    monkeypatch.setattr(torch, "empty", lambda n, **kw: Buffer(n))
    return state


def test_calls_of_one_stream_share_a_buffer(device):
    cache = {}
    a = E._ws(1000, DEV, cache, "moe_decode")
    assert E._ws(1000, DEV, cache, "moe_decode") is a and E._ws(10, DEV, cache, "moe_decode") is a
    big = E._ws(5000, DEV, cache, "moe_decode")
    assert big is not a and big.numel() >= 5000 and E._ws(1000, DEV, cache, "moe_decode") is big
    assert E._ws(1000, DEV, cache, "fp8_matmul") is not big
    assert E._ws(1000, DEV, None, "moe_decode") is not big


def test_streams_and_devices_have_buffers_of_their_own(device):
    cache = {}
    a = E._ws(1000, DEV, cache, "moe_decode")
    device["stream"] = 12
    b = E._ws(1000, DEV, cache, "moe_decode")
    assert b is not a
    device["stream"] = 11
    assert E._ws(1000, DEV, cache, "moe_decode") is a
    other = E._ws(1000, torch.device("cuda", 1), cache, "moe_decode")
    assert other is not a and E._ws(1000, DEV, cache, "moe_decode") is a


def test_a_captured_graph_shares_no_buffer(device):
    cache = {}
    a = E._ws(1000, DEV, cache, "moe_decode")
    device["capturing"] = True
    b, c = E._ws(1000, DEV, cache, "moe_decode"), E._ws(1000, DEV, cache, "moe_decode")
    assert b is not a and c is not a and b is not c
    device["capturing"] = False
    assert E._ws(1000, DEV, cache, "moe_decode") is a
