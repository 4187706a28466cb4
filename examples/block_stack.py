"""A small stack of blocks on the block-scaled FP8 operators: each block is a
projection (``fp8_block_linear``) and an MoE layer (``fp8_block_forward``), with
``norm_residual`` after each of the two: the norm of what the part gave, its gate, the
residual addition and the norm before the next part.  ``Stack`` has the projection in
the place of attention; ``AttentionStack`` has attention before it: a projection to
queries, keys and values, ``kv_append`` into the block's paged 8-bit cache and
``kv_attention`` over it.

    python examples/block_stack.py [--tokens 512] [--steps 64]

runs a prompt of that many tokens, then single tokens from a CUDA graph, for both, and
prints the times.  The weights are random.
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

    def mixed(self, i, watch=None):
        """What block i's projection takes: the normed rows."""
        return self.n

    def forward(self, x, watch=None):
        """x fp32 [T, H] -> the last norm's bf16 rows, in a buffer of the stack.
        watch(name, block, input, extra, output) is called after each part."""
        self.x.copy_(x)
        moe.norm_residual(self.x, pre_w=self.blocks[0].pre_proj, n_out=self.n)
        for i, b in enumerate(self.blocks):
            rows = self.mixed(i, watch)
            moe.fp8_block_linear(rows, *b.proj, workspace=self.proj_ws, out=self.part)
            if watch:
                watch("proj", b, rows, None, self.part)
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


class Attention:
    """One block's attention: the projection to queries, keys and values, and the cache."""

    def __init__(self, H, kv_heads, dim, n_pages, page, generator):
        self.heads, self.kv_heads, self.dim = H // dim, kv_heads, dim
        w = torch.randn((self.heads + 2 * kv_heads) * dim, H, generator=generator, device="cuda")
        self.qkv = moe.fp8_block_quantize_weights(0.02 * w)
        self.cache = moe.new_kv_cache(n_pages, kv_heads, dim, page)


class AttentionStack(Stack):
    """A stack with attention.  q_start, lengths and page_table say which sequences the
    T rows are of (``kv_append``); a decoding loop writes them on the device between
    replays of a captured ``forward``."""

    def __init__(self, blocks, attention, final_w, T, q_start, lengths, page_table, rope):
        super().__init__(blocks, final_w, T)
        a, H = attention[0], blocks[0].H
        self.attention, self.rope, self.sequences = attention, rope, (q_start, lengths, page_table)
        width = (a.heads + 2 * a.kv_heads) * a.dim
        self.qkv_ws = moe.new_workspace(moe.fp8_block_linear_workspace_size(T, width, H))
        self.kv_ws = moe.new_workspace(
            moe.kv_attention_workspace_size(lengths.shape[0], T, a.heads, a.kv_heads, a.dim))
        self.qkv = torch.empty(T, width, dtype=torch.bfloat16, device="cuda")
        self.q, self.rows = (torch.empty(T, a.heads, a.dim, dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def mixed(self, i, watch=None):
        a = self.attention[i]
        moe.fp8_block_linear(self.n, *a.qkv, workspace=self.qkv_ws, out=self.qkv)
        q, k, v = (part.unflatten(1, (-1, a.dim))
                   for part in self.qkv.split((a.heads * a.dim, a.kv_heads * a.dim, a.kv_heads * a.dim), 1))
        moe.kv_append(a.cache, k, v, *self.sequences, q=q, rope=self.rope, q_out=self.q)
        moe.kv_attention(self.q, a.cache, *self.sequences, workspace=self.kv_ws, out=self.rows)
        if watch:
            watch("attention", a, (q, k, v), self.q, self.rows)
        return self.rows.flatten(1)


def rotation(positions, dim, base=10000.0):
    """Cosines, then sines, of the angles of ``positions`` positions, formed in 64 bits."""
    turns = base ** (-torch.arange(0, dim, 2, device="cuda", dtype=torch.float64) / dim)
    angle = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * turns
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def build_attention(blocks, kv_heads=4, dim=128, n_pages=64, page=64, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [Attention(b.H, kv_heads, dim, n_pages, page, g) for b in blocks]


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
    stacks = [prompt, step]

    # the same with attention: the prompt, then tokens of the same sequence
    page = 64
    pages = -(-(a.tokens + a.steps + 8) // page)
    attention = build_attention(blocks, n_pages=pages, page=page)
    rope = rotation(pages * page, 128)

    def ints(*values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    prompt = AttentionStack(blocks, attention, final_w, a.tokens, ints(0, a.tokens), ints(a.tokens), table, rope)
    print(f"with attention, {a.tokens} tokens: {timed(lambda: prompt.forward(x), 10):.1f} us")
    length = ints(a.tokens + 1)
    step = AttentionStack(blocks, attention, final_w, 1, ints(0, 1), length, table, rope)
    graph = captured(step, token)

    def decode():
        graph.replay()
        length.add_(1)
    print(f"with attention, one token, from a graph: {timed(decode, a.steps):.1f} us")
    for s in (*stacks, prompt, step):
        for ws in (s.proj_ws, s.moe_ws, *((s.qkv_ws, s.kv_ws) if isinstance(s, AttentionStack) else ())):
            assert moe.device_error(ws) == 0
    assert all(moe.device_error(t.cache.status) == 0 for t in attention)


if __name__ == "__main__":
    main()
