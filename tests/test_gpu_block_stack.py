"""The block-scaled operators together, as examples/block_stack.py runs them: every
part against its plain 64-bit form on the input it had, and the whole from a graph."""
import importlib.util
import os

import pytest
import torch

import block_reference as ref
import test_gpu_block as block
import test_gpu_norm as norm
import w8a8_quantised_moe_gb300 as moe

pytestmark = pytest.mark.gpu


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "block_stack.py")
    spec = importlib.util.spec_from_file_location("block_stack", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def check_part(name, b, before, extra, after):
    if name == "proj":
        want, mag = ref.linear(before, *b.proj)
        bound = block.SUM_REL * mag * (1 + block.BF16) + block.BF16 * want.abs() + 2.0**-134
        assert ((after.double() - want).abs() <= bound).all()
    elif name == "norm":
        branch, post_w, gate, pre_w = extra
        norm.check(dict(x=before, branch=branch, post_w=post_w, gate=gate, scale=0.5, pre_w=pre_w, eps=1e-6), after)
    else:
        want = ref.moe(before, b.router_w, None, *b.w13, *b.w2, b.top_k).bfloat16().double()
        top = (before.double() @ b.router_w.double()).topk(b.top_k + 1, dim=1).values
        clear = top[:, b.top_k - 1] - top[:, b.top_k] > 1e-3  # the choice of experts hangs on no rounding
        assert clear.any()
        err = (after.double() - want).abs()[clear]
        assert err.max() <= block.Y_MAX_REL * want.abs().max()
        assert err.sum() <= block.Y_MEAN_REL * want[clear].abs().sum()


@pytest.mark.parametrize("T", [1, 5, 70, 600])
def test_each_part_of_the_stack(T):
    ex = example()
    blocks, final_w = ex.build(H=512, I=256, E=8, top_k=2, n_blocks=2, seed=T)
    stack = ex.Stack(blocks, final_w, T)
    x = torch.randn(T, 512, generator=block.gen(T), device="cuda")
    seen = []

    def watch(name, *what):
        check_part(name, *what)
        seen.append(name)
    out = stack.forward(x, watch).clone()
    assert seen == ["proj", "norm", "moe", "norm"] * 2
    assert torch.equal(stack.forward(x), out)  # the same bits without the checks between
    assert moe.device_error(stack.proj_ws) == 0 and moe.device_error(stack.moe_ws) == 0


@pytest.mark.parametrize("T", [1, 40])
def test_the_stack_from_a_graph(T):
    ex = example()
    blocks, final_w = ex.build(H=512, I=256, E=8, top_k=2, n_blocks=3, seed=3)
    stack = ex.Stack(blocks, final_w, T)
    x = torch.randn(T, 512, generator=block.gen(1), device="cuda")
    graph = ex.captured(stack, x)
    for seed in (2, 3):
        x.copy_(torch.randn(T, 512, generator=block.gen(seed), device="cuda"))
        want = stack.forward(x).clone()
        stack.n.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(stack.n, want)
