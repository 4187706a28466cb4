"""One workspace, sized for the largest batch, for calls of fewer tokens too."""
import pytest
import torch

import test_gpu_block as block
import w8a8_quantised_moe_gb300 as moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,I,E,k,steps", [(2048, 768, 8, 2, (9, 8, 1, 7)), (1024, 256, 8, 1, (12, 8, 9, 1)),
                                           (1024, 256, 64, 2, (129, 128, 40, 8, 129, 3))])
def test_block_layer(H, I, E, k, steps):
    layer = block.Layer(max(steps), H, I, E, k, seed=H)
    ws = moe.new_workspace(moe.fp8_block_workspace_size(max(steps), H, I, E, k))
    x, *rest = layer.args()
    for T in steps:
        want = moe.fp8_block_forward(x[:T], *rest)
        assert torch.equal(moe.fp8_block_forward(x[:T], *rest, workspace=ws), want), T
        assert moe.device_error(ws) == 0


def int8_layer(T, H, I, E, k):
    g = block.gen(T)
    x, router_w = block.activations(g, T, H), torch.randn(H, E, generator=g, device="cuda") / H**0.5
    w13, s13 = moe.quantize_weights(torch.randn(E * 2 * I, H, generator=g, device="cuda"))
    w2, s2 = moe.quantize_weights(torch.randn(E * H, I, generator=g, device="cuda"))
    return x, (router_w, None, w13.view(E, 2 * I, H), s13.view(E, 2 * I), w2.view(E, H, I), s2.view(E, H), k)


def test_int8_layer():
    x, rest = int8_layer(129, 512, 256, 64, 2)
    ws = moe.new_workspace(moe.workspace_size(129, 512, 256, 64, 2))
    for T in (129, 128, 5):
        assert torch.equal(moe.forward(x[:T], *rest, workspace=ws), moe.forward(x[:T], *rest)), T
