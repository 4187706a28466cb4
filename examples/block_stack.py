"""A small stack of blocks on the block-scaled FP8 operators: each block is a
projection (``fp8_block_linear``, here in the place of attention's) and an MoE layer
(``fp8_block_forward``), with ``norm_residual`` after each of the two: the norm of
what the part gave, its gate, the residual addition and the norm before the next part.

    python examples/block_stack.py [--tokens 512] [--steps 64]

runs a prompt of that many tokens, then single tokens from a CUDA graph, and prints
the times.  The weights are random.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import w8a8_quantised_moe_gb300 as moe  # noqa: E402


class Block:
    """One block's weights, quantised once."""

    def __init__(self, H, I, E, top_k, generator):
        def r(*shape):
            return torch.randn(*shape, generator=generator, device="cuda")

        def near_one():
            return (1 + 0.1 * r(H)).bfloat16()
        self.top_k, self.H, self.I, self.E = top_k, H, I, E
        self.proj = moe.fp8_block_quantize_weights(0.02 * r(H, H))
        self.w13 = moe.fp8_block_quantize_weights(0.02 * r(E, 2 * I, H))
        self.w2 = moe.fp8_block_quantize_weights(0.02 * r(E, H, I))
        self.router_w = r(H, E) / H**0.5
        self.pre_proj, self.post_proj, self.pre_moe, self.post_moe = (near_one() for _ in range(4))
        self.gate = near_one()


class Stack:
    """Blocks and the buffers of a batch of T tokens, kept between calls."""

    def __init__(self, blocks, final_w, T):
        b = blocks[0]
        self.blocks, self.final_w, self.T = blocks, final_w, T
        self.proj_ws = moe.new_workspace(moe.fp8_block_linear_workspace_size(T, b.H, b.H))
        self.moe_ws = moe.new_workspace(moe.fp8_block_workspace_size(T, b.H, b.I, b.E, b.top_k))
        self.x = torch.empty(T, b.H, dtype=torch.float32, device="cuda")  # the residual stream, in binary32
        self.n, self.part = (torch.empty(T, b.H, dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def forward(self, x, watch=None):
        """x fp32 [T, H] -> the last norm's bf16 rows, in a buffer of the stack.
        watch(name, block, input, extra, output) is called after each part."""
        self.x.copy_(x)
        moe.norm_residual(self.x, pre_w=self.blocks[0].pre_proj, n_out=self.n)
        for i, b in enumerate(self.blocks):
            moe.fp8_block_linear(self.n, *b.proj, workspace=self.proj_ws, out=self.part)
            if watch:
                watch("proj", b, self.n, None, self.part)
            before = self.x.clone() if watch else None
            moe.norm_residual(self.x, self.part, post_w=b.post_proj, gate=b.gate, scale=0.5, pre_w=b.pre_moe,
                              x_out=self.x, n_out=self.n)
            if watch:
                watch("norm", b, before, (self.part, b.post_proj, b.gate, b.pre_moe), (self.x, self.n))
            moe.fp8_block_forward(self.n, b.router_w, None, *b.w13, *b.w2, b.top_k, workspace=self.moe_ws,
                                  out=self.part)
            if watch:
                watch("moe", b, self.n, None, self.part)
            next_w = self.blocks[i + 1].pre_proj if i + 1 < len(self.blocks) else self.final_w
            before = self.x.clone() if watch else None
            moe.norm_residual(self.x, self.part, post_w=b.post_moe, gate=b.gate, scale=0.5, pre_w=next_w,
                              x_out=self.x, n_out=self.n)
            if watch:
                watch("norm", b, before, (self.part, b.post_moe, b.gate, next_w), (self.x, self.n))
        return self.n


def build(H=2048, I=768, E=32, top_k=4, n_blocks=4, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    blocks = [Block(H, I, E, top_k, g) for _ in range(n_blocks)]
    return blocks, (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).bfloat16()


def captured(stack, x):
    """A CUDA graph of stack.forward on the buffer x (run once before)."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        stack.forward(x)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        stack.forward(x)
    return graph


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--steps", type=int, default=64)
    a = ap.parse_args()
    blocks, final_w = build()
    H = blocks[0].H

    def timed(f, n):
        f()
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        begin.record()
        for _ in range(n):
            f()
        end.record()
        end.synchronize()
        return begin.elapsed_time(end) / n * 1e3

    prompt = Stack(blocks, final_w, a.tokens)
    x = torch.randn(a.tokens, H, device="cuda")
    print(f"{len(blocks)} blocks, {a.tokens} tokens: {timed(lambda: prompt.forward(x), 10):.1f} us")
    step = Stack(blocks, final_w, 1)
    token = x[-1:].clone()
    graph = captured(step, token)
    print(f"{len(blocks)} blocks, one token, from a graph: {timed(graph.replay, a.steps):.1f} us")
    for s in (prompt, step):
        for ws in (s.proj_ws, s.moe_ws):
            assert moe.device_error(ws) == 0


if __name__ == "__main__":
    main()
