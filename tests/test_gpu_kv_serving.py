"""The paged cache as a serving loop uses it: a prompt, tokens from a graph, other streams,
a wait that runs out; and the operators together in examples/block_stack.py."""
import pytest
import torch

import kv_reference as ref
import test_gpu_block_stack as stack
import test_gpu_stream_allocations as streams
import w8a8_quantised_moe_gb300 as moe
from test_gpu_kv_append import rows
from test_gpu_kv_attention import MANY, ONE, queries

pytestmark = pytest.mark.gpu

PAGE, DIM = 16, 64


def attention_stack(ex, blocks, final_w, attention, seqs, table, T):
    starts = [0]
    for n, _ in seqs:
        starts.append(starts[-1] + n)
    def ints(v):
        return torch.tensor(v, dtype=torch.int32).cuda()
    return ex.AttentionStack(blocks, attention, final_w, T, ints(starts), ints([length for _, length in seqs]), table,
                             ex.rotation(200, DIM))


@pytest.mark.parametrize("T", [1, 5, 90])
def test_each_part_of_a_stack_with_attention(T):
    """A prompt of T tokens after 40 cached ones, and a second sequence of one token."""
    ex = stack.example()
    blocks, final_w = ex.build(H=512, I=256, E=8, top_k=2, n_blocks=2, seed=T)
    attention = ex.build_attention(blocks, kv_heads=2, dim=DIM, n_pages=20, page=PAGE)
    seqs = [(T, 40 + T), (1, 33)]
    batch = ref.Batch(seqs, PAGE, n_pages=20, seed=T)
    for a in attention:
        a.cache = ref.filled_cache(batch, 2, DIM, T)
    s = attention_stack(ex, blocks, final_w, attention, seqs, batch.args[2], T + 1)
    stored = {id(a): ref.Stored(a.cache) for a in attention}
    seen = []

    def watch(name, part, before, extra, after):
        seen.append(name)
        if name != "attention":
            return stack.check_part(name, part, before, extra, after)
        q, k, v = before
        stored[id(part)].append(k, v, batch, s.rope)
        stored[id(part)].check(part.cache)
        ref.check_queries(q, extra, batch, s.rope, False)
        ref.check_attention(extra, part.cache, batch, after)
    x = torch.randn(T + 1, 512, generator=torch.Generator(device="cuda").manual_seed(T), device="cuda")
    out = s.forward(x, watch).clone()
    assert seen == ["attention", "proj", "norm", "moe", "norm"] * 2
    assert torch.equal(s.forward(x), out)  # tokens stored twice are stored the same
    for ws in (s.qkv_ws, s.kv_ws, *(a.cache.status for a in attention)):
        assert moe.device_error(ws) == 0


def test_tokens_of_two_sequences_from_a_graph():
    ex = stack.example()
    blocks, final_w = ex.build(H=512, I=256, E=8, top_k=2, n_blocks=2, seed=7)
    pages = 20
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).int().view(2, 10).cuda()
    results = []
    for replayed in (False, True):
        attention = ex.build_attention(blocks, kv_heads=2, dim=DIM, n_pages=pages, page=PAGE)
        prompt = attention_stack(ex, blocks, final_w, attention, [(50, 50), (7, 7)], table, 57)
        prompt.forward(torch.randn(57, 512, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda"))
        step = attention_stack(ex, blocks, final_w, attention, [(1, 51), (1, 8)], table, 2)
        token, lengths = torch.zeros(2, 512, device="cuda"), step.sequences[1]
        graph = ex.captured(step, token) if replayed else None
        outs = []
        for i in range(24):
            token.copy_(torch.randn(2, 512, generator=torch.Generator(device="cuda").manual_seed(10 + i), device="cuda"))
            if replayed:
                graph.replay()
            else:
                # the captured stack has stored one token of zeros at the first place while it was warmed up
                if i == 0:
                    kept = token.clone()
                    step.forward(torch.zeros_like(token))
                    token.copy_(kept)
                step.forward(token)
            outs.append(step.n.clone())
            lengths.add_(1)
        results.append((torch.stack(outs), [a.cache for a in attention]))
    assert torch.equal(results[0][0], results[1][0])
    for a, b in zip(results[0][1], results[1][1]):
        for name in ("k", "v", "k_scale", "v_scale"):
            assert torch.equal(getattr(a, name), getattr(b, name)), name


@pytest.mark.parametrize("seqs", [ONE, MANY], ids=["one", "many"])
def test_on_another_stream_while_the_current_one_is_busy(seqs):
    batch = ref.Batch(seqs, 32, seed=1)
    cache = ref.filled_cache(batch, 2, 64, 1)
    q, k, v = queries(batch.T, 6, 64, 1), rows(batch.T, 2, 64, 2), rows(batch.T, 2, 64, 3)
    rope = ref.rope_table(max(length for _, length in seqs), 64)
    streams.check(lambda **kw: (moe.kv_append(cache, k, v, *batch.args, q=q, rope=rope, **kw),), q.nbytes)
    need = moe.kv_attention_workspace_size(len(seqs), batch.T, 6, 2, 64)
    streams.check(lambda **kw: (moe.kv_attention(q, cache, *batch.args, **kw),), need, q.nbytes)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("seqs", [MANY, [(700, 900)], [(40, 40)] * 9], ids=["many", "prompt", "short"])
def test_a_wait_that_runs_out_then_the_same_results_again(monkeypatch, seqs, dim):
    batch = ref.Batch(seqs, 16, seed=2)
    cache = ref.filled_cache(batch, 2, dim, 2)
    q = queries(batch.T, 8, dim, 2)
    ws = moe.new_workspace(moe.kv_attention_workspace_size(len(seqs), batch.T, 8, 2, dim))
    ws[256:] = 0x7F  # what the parts' places hold may be anything
    monkeypatch.setenv("MOE_INJECT", "stall")
    moe.set_wait_timeout_ns(2_000_000)
    try:
        out = moe.kv_attention(q, cache, *batch.args, workspace=ws)
        assert moe.device_error(ws) == -5
    finally:
        monkeypatch.delenv("MOE_INJECT")
        moe.set_wait_timeout_ns(0)
    assert moe.device_error(ws) == 0
    got = moe.kv_attention(q, cache, *batch.args, workspace=ws, out=out)
    assert moe.device_error(ws) == 0
    ref.check_attention(q, cache, batch, got)


def test_the_same_bits_when_the_last_call_is_still_running():
    """Calls one behind the other share a workspace; each waits for the parts of the one before."""
    batches = [ref.Batch(seqs, 16, n_pages=400, seed=3) for seqs in (MANY, ONE, [(300, 2000)])]
    caches = [ref.filled_cache(b, 2, 64, 3) for b in batches]
    qs = [queries(b.T, 4, 64, 3) for b in batches]
    ws = moe.new_workspace(max(moe.kv_attention_workspace_size(len(b.seqs), b.T, 4, 2, 64) for b in batches))
    want = [moe.kv_attention(q, c, *b.args).clone() for q, c, b in zip(qs, caches, batches)]
    torch.cuda.synchronize()
    outs = [[moe.kv_attention(q, c, *b.args, workspace=ws) for q, c, b in zip(qs, caches, batches)] for _ in range(10)]
    torch.cuda.synchronize()
    for got in outs:
        assert all(torch.equal(a, b) for a, b in zip(got, want))
