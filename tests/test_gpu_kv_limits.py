"""The paged cache at the limits of what its calls are told: tokens behind the page table."""
import pytest
import torch

import kv_reference as ref
import w8a8_quantised_moe_gb300 as moe
from test_gpu_kv_append import rows

pytestmark = pytest.mark.gpu

INT_MAX = 2**31 - 1


@pytest.mark.parametrize("over", [1, "some", "all", "past", INT_MAX])
@pytest.mark.parametrize("n", [1, 5, 40, 130])
@pytest.mark.parametrize("page,dim", [(16, 64), (64, 128)])
def test_tokens_behind_the_page_table_are_left_out(page, dim, n, over):
    """A sequence `over` tokens longer than its pages: those tokens are not stored and their queries left
    alone, what the pages hold stays, the others are stored where they belong, and the error word is set."""
    cap = 4 * page
    over = {"some": (n + 1) // 2, "all": n, "past": n + 3}.get(over, over)
    batch = ref.Batch([(2, 20), (n, cap), (0, 9), (1, page + 1)], page, extra_pages=0)
    assert batch.table.shape[1] == 4
    length = min(cap + over, INT_MAX)
    batch.args[1][1] = length
    cache = ref.filled_cache(batch, 2, dim)
    want = ref.Stored(cache)
    k, v, q = (rows(batch.T, h, dim, i) for i, h in enumerate((2, 2, 6)))
    rope = ref.rope_table(cap, dim)
    out = torch.full((batch.T, 6, dim), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.kv_append(cache, k, v, *batch.args, q=q, rope=rope, q_out=out)
    stored = max(0, n - (length - cap))
    batch.seqs[1] = (stored, cap)  # the rows stay where they are
    want.append(k, v, batch, rope)
    want.check(cache)
    ref.check_queries(q, out, batch, rope, False)
    assert (out[batch.starts[1] + stored:batch.starts[2]] == 7).all()
    assert moe.device_error(cache.status) == -7 and moe.device_error(cache.status) == 0
    # the same without queries and without rotation
    want.append(k, v, batch)
    assert moe.kv_append(cache, k, v, *batch.args) is None
    want.check(cache)
    assert moe.device_error(cache.status) == -7


def test_a_decoding_loop_that_runs_past_its_pages():
    """From a graph: every token that fits is as it was after the last one that did."""
    page, dim, cap = 16, 64, 48
    cache = moe.new_kv_cache(6, 2, dim, page)
    table = torch.tensor([[3, 1, 5], [0, 4, 2]], dtype=torch.int32, device="cuda")
    q_start = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    lengths = torch.tensor([1, 1], dtype=torch.int32, device="cuda")
    k, v = rows(2, 2, dim, 1), rows(2, 2, dim, 2)
    rope = ref.rope_table(64, dim)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        moe.kv_append(cache, k, v, q_start, lengths, table, rope=rope)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.kv_append(cache, k, v, q_start, lengths, table, rope=rope)
    for step in range(cap):
        k.copy_(rows(2, 2, dim, 10 * step))
        graph.replay()
        lengths += 1
    assert moe.device_error(cache.status) == 0
    full = [getattr(cache, name).clone() for name in ("k", "v", "k_scale", "v_scale")]
    for step in range(5):
        k.copy_(rows(2, 2, dim, 10 * step + 1, size=64.0))
        graph.replay()
        lengths += 1
    assert moe.device_error(cache.status) == -7
    for name, was in zip(("k", "v", "k_scale", "v_scale"), full):
        assert torch.equal(getattr(cache, name), was), name
