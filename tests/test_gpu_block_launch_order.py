"""Launches of the linear layer back to back whose tensor memory would not fit one SM together."""
import pytest
import torch

import test_gpu_block as block
import w8a8_quantised_moe_gb300 as moe

pytestmark = pytest.mark.gpu

ROWS = (100, 1, 128, 16, 65, 30, 128, 1, 60, 100, 8)


def test_few_rows_back_to_back_on_two_streams():
    g = block.gen(1)
    w_q, w_s = block.weight(g, 2048, 2048)
    x = {M: block.activations(g, M, 2048) for M in ROWS}
    want = {M: moe.fp8_block_linear(x[M], w_q, w_s) for M in ROWS}
    streams = [torch.cuda.current_stream(), torch.cuda.Stream()]
    streams[1].wait_stream(streams[0])
    ws = [moe.new_workspace(moe.fp8_block_linear_workspace_size(128, 2048, 2048)) for _ in streams]
    outs = [[torch.empty_like(want[M]) for M in ROWS * 4] for _ in streams]
    torch.cuda.synchronize()
    for i, M in enumerate(ROWS * 4):
        for s, w, o in zip(streams, ws, outs):
            moe.fp8_block_linear(x[M], w_q, w_s, workspace=w, out=o[i], stream=s)
    torch.cuda.synchronize()
    for w, o in zip(ws, outs):
        assert moe.device_error(w) == 0
        assert all(torch.equal(y, want[M]) for y, M in zip(o, ROWS * 4))
