"""Which device the mixer's calls run on (no GPU: the streams are stand-ins)."""
from types import SimpleNamespace

import torch

from selective_state_space_83_amd import mixer


def test_a_given_stream_names_its_own_device(monkeypatch):
    """A stream of another device than the current one: the call's tensors have to
    lie on the stream's."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    stream = SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=7)
    assert mixer._current(stream) == (1, 7)


def test_without_a_stream_the_current_device(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 2)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 10 + dev, raising=False)
    assert mixer._current(None) == (2, 12)
