"""The stream that the binding passes on, without a GPU."""

import types

import torch

import combine_ep_dispatch_amd as epx


def test_current_stream_with_and_without_the_raw_call(monkeypatch):
    """torch's raw handle of the current stream is a private call: without it the
    public one serves."""
    dev = torch.device("cuda:3")
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 100 + index, raising=False)
    assert epx._stream(None, dev) == 103
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: types.SimpleNamespace(cuda_stream=200 + d.index))
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
    assert epx._stream(None, dev) == 203


def test_given_streams_are_passed_on():
    dev = torch.device("cuda:0")
    assert epx._stream(17, dev) == 17
    assert epx._stream(types.SimpleNamespace(cuda_stream=19), dev) == 19
