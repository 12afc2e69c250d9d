"""The stream that a call without one runs on is PyTorch's current stream, whichever way the
binding reads it."""
from __future__ import annotations

import types

import pytest
import torch

import mixture_experts_ffn_renorm_gb300 as m

PRIVATE = ("_cuda_getCurrentRawStream", "_cuda_getDevice")


@pytest.fixture(autouse=True)
def _fresh(monkeypatch):
    monkeypatch.setattr(m, "_current_stream", None)


@pytest.mark.parametrize("missing", [(), *[(p,) for p in PRIVATE], PRIVATE])
def test_chosen_by_what_pytorch_has(monkeypatch, missing):
    # fakes: no GPU needed
    state = {"device": 0}
    streams = {0: 0x1000, 1: 0x2000}
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda *a: types.SimpleNamespace(cuda_stream=streams[state["device"]]))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: streams[d], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: state["device"], raising=False)
    for name in missing:
        monkeypatch.delattr(torch._C, name)
    for device, at in ((0, 0x1000), (1, 0x2000), (0, 0x3000)):
        state["device"], streams[device] = device, at    # read anew at each call
        assert m._stream(None) == at
    assert m._stream(5) == 5 and m._stream(types.SimpleNamespace(cuda_stream=7)) == 7


@pytest.mark.gpu
@pytest.mark.parametrize("missing", [False, True])
def test_follows_the_current_stream(monkeypatch, missing):
    if missing:
        monkeypatch.delattr(torch._C, PRIVATE[0])
    assert m._stream(None) == torch.cuda.current_stream().cuda_stream
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert m._stream(None) == side.cuda_stream != 0
    assert m._stream(None) == torch.cuda.current_stream().cuda_stream
