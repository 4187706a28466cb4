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


SHAPES = [(2048, 768, 8, 2), (4096, 1536, 64, 2), (4096, 1536, 2, 1), (1024, 256, 8, 1), (7168, 2048, 256, 8),
          (128, 128, 256, 8), (16384, 128, 130, 4), (1408, 640, 1, 1), (4096, 256, 33, 5)]


@pytest.fixture(scope="module")
def lib():
    from w8a8_quantised_moe_gb300 import build
    build.build()
    return _lib.load()


@pytest.mark.parametrize("size", ["moe_w8a8_workspace_size", "moe_w8a8_fp8_block_workspace_size"])
@pytest.mark.parametrize("shape", SHAPES)
def test_a_workspace_for_more_tokens_serves_fewer(lib, size, shape):
    need = [getattr(lib, size)(T, *shape) for T in [*range(0, 6000), 1 << 16, (1 << 16) + 1, 1 << 20]]
    assert need[0] > 0 and all(a <= b for a, b in zip(need, need[1:]))


def test_a_linear_workspace_for_more_rows_serves_fewer(lib):
    for size in (lib.moe_w8a8_linear_workspace_size, lib.moe_w8a8_fp8_block_linear_workspace_size):
        for N, K in ((128, 128), (4096, 4096)):
            need = [size(M, N, K) for M in range(0, 3000)]
            assert need[0] > 0 and all(a <= b for a, b in zip(need, need[1:]))
