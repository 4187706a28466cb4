"""What a call allocates belongs to the stream it is given (CPU: the library and the
streams are stand-ins).  Memory of another stream's pool can still be in use there, and
a workspace zeroed there can be zeroed after the call's kernels have written to it."""
import contextlib

import pytest
import torch

import w8a8_quantised_moe_gb300 as moe
from w8a8_quantised_moe_gb300 import _lib

T, H, I, E, K = 4, 128, 128, 2, 1


class FakeLibrary:
    def __getattr__(self, name):
        def call(*args):
            return 4096 if name.endswith("workspace_size") else 0
        return call


class FakeStream:
    cuda_stream = 7


@pytest.fixture
def allocations(monkeypatch):
    """[(function, stream it ran under)] of torch.empty, zeros and empty_like."""
    seen, under = [], [None]

    @contextlib.contextmanager
    def stream(s):
        under.append(s)
        yield
        under.pop()

    def watched(name, real):
        def call(*args, **kw):
            kw.pop("device", None)
            seen.append((name, under[-1]))
            return real(*args, **kw)
        return call
    monkeypatch.setattr(_lib, "load", lambda: FakeLibrary())
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(moe, "_need", lambda *a: None)
    monkeypatch.setattr(moe, "_fits", lambda *a: True)
    monkeypatch.setattr(moe, "_raw_stream", lambda stream, t: 0)
    monkeypatch.setattr(moe, "_stream", lambda stream: 0)
    monkeypatch.setattr(moe, "_room", lambda workspace: (0, workspace.nbytes))
    for name in ("empty", "zeros", "empty_like"):
        monkeypatch.setattr(torch, name, watched(name, getattr(torch, name)))
    return seen


def layer(codes, blocks):
    def scale(rows, cols):
        return torch.ones(E, rows // 128, cols // 128) if blocks else torch.ones(E, rows)
    return (torch.ones(T, H, dtype=torch.bfloat16), torch.ones(H, E), None, torch.ones(E, 2 * I, H, dtype=codes),
            scale(2 * I, H), torch.ones(E, H, I, dtype=codes), scale(H, I))


X = torch.ones(T, H, dtype=torch.bfloat16)
W = torch.ones(H)
S8, U8 = torch.int8, torch.uint8
CALLS = {
    "quantize_weights": lambda **kw: moe.quantize_weights(torch.ones(16, H), **kw),
    "quantize_weights_smoothed": lambda **kw: moe.quantize_weights_smoothed(torch.ones(16, H), W, **kw),
    "fp8_quantize_weights": lambda **kw: moe.fp8_quantize_weights(torch.ones(16, H), **kw),
    "forward": lambda **kw: moe.forward(*layer(S8, False), K, **kw),
    "forward_debug": lambda **kw: moe.forward_debug(*layer(S8, False), K, **kw),
    "forward_fused": lambda **kw: moe.forward_fused(*layer(S8, False), K, fields=None, **kw),
    "forward_smooth": lambda **kw: moe.forward_smooth(*layer(S8, False)[:3], torch.ones(E, H), *layer(S8, False)[3:], K,
                                                      fields=None, **kw),
    "linear": lambda **kw: moe.linear(X, torch.ones(16, H, dtype=S8), torch.ones(16), **kw),
    "fp8_forward": lambda **kw: moe.fp8_forward(*layer(U8, False), K, **kw),
    "fp8_forward_debug": lambda **kw: moe.fp8_forward_debug(*layer(U8, False), K, **kw),
    "fp8_block_quantize_weights": lambda **kw: moe.fp8_block_quantize_weights(torch.ones(16, H), **kw),
    "fp8_block_linear": lambda **kw: moe.fp8_block_linear(X, torch.ones(16, H, dtype=U8), torch.ones(1, 1), **kw),
    "fp8_block_forward": lambda **kw: moe.fp8_block_forward(*layer(U8, True), K, **kw),
    "norm_residual": lambda **kw: moe.norm_residual(X, X, pre_w=W, **kw),
    "norm_residual, norm only": lambda **kw: moe.norm_residual(X, pre_w=W, **kw),
}


@pytest.mark.parametrize("name", CALLS)
def test_a_call_allocates_on_its_stream(name, allocations):
    CALLS[name]()
    plain = [n for n, _ in allocations]
    assert plain and all(s is None for _, s in allocations)
    del allocations[:]
    s = FakeStream()
    CALLS[name](stream=s)
    assert [n for n, _ in allocations] == plain
    assert all(under is s for _, under in allocations)


def test_host_forward_allocates_on_its_stream(allocations, monkeypatch):
    monkeypatch.setattr(moe, "_need_host", lambda *a: None)
    s = FakeStream()
    x, *rest = layer(S8, False)
    moe.forward_host(x, *rest, K, y_host=x.clone(), stream=s)
    assert [n for n, _ in allocations] == ["empty", "empty", "zeros"]
    assert all(under is s for _, under in allocations)


def test_a_call_with_its_buffers_given_allocates_nothing(allocations):
    ws = torch.ones(4096, dtype=U8)
    s = FakeStream()
    CALLS["fp8_block_linear"](stream=s, workspace=ws, out=torch.ones(T, 16, dtype=torch.bfloat16))
    CALLS["fp8_block_forward"](stream=s, workspace=ws, out=X.clone())
    CALLS["norm_residual"](stream=s, x_out=X.clone(), n_out=X.clone())
    assert allocations == []
