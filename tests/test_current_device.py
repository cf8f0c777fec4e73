"""The stream that a call launches on belongs to the GPU of its tensors.  CPU only."""
import pytest
import torch

import group_sparse_swiglu_amd as E


@pytest.fixture
def gpu(monkeypatch):
    state = dict(current=0, streams={0: 0, 1: 0})
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: state["streams"][i], raising=False)
    monkeypatch.setattr(E, "_several_gpus", lambda: True, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: state["current"], raising=False)
    return state


def test_default_stream_of_another_gpu_is_refused(gpu):
    assert E._stream(torch.device("cuda", 0)) == 0
    with pytest.raises(E.EsgError, match="cuda:1"):
        E._stream(torch.device("cuda", 1))
    gpu["current"] = 1
    assert E._stream(torch.device("cuda", 1)) == 0
    with pytest.raises(E.EsgError, match="cuda:0"):
        E._stream(torch.device("cuda", 0))


def test_own_streams_name_their_gpu(gpu):
    gpu["streams"][1] = 77
    assert E._stream(torch.device("cuda", 1)) == 77
