"""Workspaces as a serving loop keeps them (CPU: nothing is launched)."""
import pytest
import torch

import test_stream_allocations as calls
import w8a8_quantised_moe_gb300 as moe
from w8a8_quantised_moe_gb300 import _lib


@pytest.fixture
def no_library(monkeypatch):
    monkeypatch.setattr(_lib, "load", lambda: calls.FakeLibrary())
    monkeypatch.setattr(moe, "_need", lambda *a: None)
    monkeypatch.setattr(moe, "_fits", lambda *a: True)
    monkeypatch.setattr(moe, "_raw_stream", lambda stream, t: 0)
    monkeypatch.setattr(moe, "_stream", lambda stream: 0)


@pytest.mark.parametrize("name", [n for n in calls.CALLS if "quantize" not in n and "norm" not in n])
def test_a_workspace_in_host_memory_is_refused(name, no_library):
    with pytest.raises(ValueError, match="workspace: expected a contiguous cuda tensor"):
        calls.CALLS[name](workspace=torch.zeros(4096, dtype=torch.uint8))


def test_a_strided_workspace_is_refused():
    class OnGpu:
        is_cuda, device, shape = True, "cuda:0", (2048,)
        is_contiguous, stride = staticmethod(lambda: False), staticmethod(lambda: (0,))
    with pytest.raises(ValueError, match="workspace: expected a contiguous cuda tensor"):
        moe._room(OnGpu())
