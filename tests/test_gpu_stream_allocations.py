"""Calls on another stream than the current one, without buffers: complete and right
while the current stream is still busy, on memory that it left dirty."""
import pytest
import torch

import test_gpu_block as block
import w8a8_quantised_moe_gb300 as moe

pytestmark = pytest.mark.gpu


def dirty_pool(nbytes):
    """Blocks of these sizes, full of ones, back in the current stream's pool."""
    held = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in nbytes for _ in range(2)]
    torch.cuda.synchronize()
    del held


def check(call, *nbytes):
    want = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    first = call(stream=side)  # loads what runs below and fills the stream's pool
    with torch.cuda.stream(side):
        assert all(torch.equal(a, b) for a, b in zip(first, want) if a is not None)
    del first
    dirty_pool(nbytes)
    torch.cuda._sleep(400_000_000)  # a fifth of a second of the current stream
    got = call(stream=side)
    with torch.cuda.stream(side):
        equal = [torch.equal(a, b) for a, b in zip(got, want) if a is not None]
    busy = not torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    assert busy and all(equal)
    assert all(torch.equal(a, b) for a, b in zip(got, want) if a is not None)


@pytest.mark.parametrize("M", [3, 40, 200])
def test_linear(M):
    g = block.gen(M)
    x, (w_q, w_s) = block.activations(g, M, 512), block.weight(g, 256, 512)
    check(lambda **kw: (moe.fp8_block_linear(x, w_q, w_s, **kw),), moe.fp8_block_linear_workspace_size(M, 256, 512),
          M * 256 * 2)


@pytest.mark.parametrize("shape", [(3, 512, 256, 8, 2), (40, 512, 256, 64, 2), (300, 512, 256, 8, 2)])
def test_layer(shape):
    layer = block.Layer(*shape, seed=1)
    check(lambda **kw: (moe.fp8_block_forward(*layer.args(), **kw),), moe.fp8_block_workspace_size(*shape),
          layer.x.nbytes)


def test_norm_and_weight_quantiser():
    g = block.gen(2)
    x, branch = block.activations(g, 200, 512), block.activations(g, 200, 512)
    w = torch.randn(512, 512, generator=g, device="cuda")
    check(lambda **kw: moe.norm_residual(x, branch, pre_w=x[0], **kw), x.nbytes)
    check(lambda **kw: moe.fp8_block_quantize_weights(w, **kw), w.numel())
    check(lambda **kw: moe.quantize_weights(w, **kw), w.numel())


def test_int8_forms():
    """(Not the one-kernel layer: its launch takes the whole GPU at once, so it waits for the other stream.)"""
    g = block.gen(3)
    T, H, I, E, k = 40, 512, 256, 8, 2
    x, router_w = block.activations(g, T, H), torch.randn(H, E, generator=g, device="cuda") / H**0.5
    w13, s13 = moe.quantize_weights(torch.randn(E * 2 * I, H, generator=g, device="cuda"))
    w2, s2 = moe.quantize_weights(torch.randn(E * H, I, generator=g, device="cuda"))
    args = x, router_w, None, w13.view(E, 2 * I, H), s13.view(E, 2 * I), w2.view(E, H, I), s2.view(E, H), k
    ws = moe.workspace_size(T, H, I, E, k)
    check(lambda **kw: (moe.forward(*args, **kw),), ws, x.nbytes)
    check(lambda **kw: (moe.linear(x, w13, s13, **kw),), moe.linear_workspace_size(T, E * 2 * I, H))
