"""The paged cache at the limits of what its calls are told: tokens behind the page table, pages
behind the window, scales that are not finite, scores of thousands, bad pages."""
import math

import pytest
import torch

import block_reference as block
import kv_reference as ref
import w8a8_quantised_moe_gb300 as moe
from test_gpu_kv_append import rows
from test_gpu_kv_attention import queries

pytestmark = pytest.mark.gpu

INT_MAX = 2**31 - 1


def space(batch, q_heads, cache):
    return moe.new_workspace(
        moe.kv_attention_workspace_size(len(batch.seqs), batch.T, q_heads, cache.heads, cache.dim))


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


def behind(batch, window):
    """[first key that a row of the sequence sees]"""
    return [max(0, length - n - window + 1) if window else 0 for n, length in batch.seqs]


WINDOWED = [[(1, 700), (1, 300), (1, 40)], [(6, 701), (3, 299)], [(100, 702), (70, 300), (1, 500)]]


@pytest.mark.parametrize("window", [1, 17, 100, 129])
@pytest.mark.parametrize("seqs", WINDOWED, ids=["one", "few", "many"])
@pytest.mark.parametrize("page,dim", [(16, 64), (64, 128), (128, 64)])
def test_pages_behind_the_window_are_not_asked_for(page, dim, seqs, window):
    """A serving loop takes pages back that no row sees any more: their entries are no pages, and no error."""
    batch = ref.Batch(seqs, page, seed=20)
    cache = ref.filled_cache(batch, 2, dim, 20)
    q = queries(batch.T, 8, dim, 20)
    ws = space(batch, 8, cache)
    lse = torch.empty(batch.T, 8, device="cuda")
    want = moe.kv_attention(q, cache, *batch.args, window=window, workspace=ws, lse=lse)
    ref.check_attention(q, cache, batch, want, lse, window=window)
    assert moe.device_error(ws) == 0
    table, taken = batch.args[2].clone(), 0
    for b, first in enumerate(behind(batch, window)):
        table[b, :first // page] = -1
        taken += first // page
    assert taken > 0
    got = moe.kv_attention(q, cache, *batch.args[:2], table, window=window, workspace=ws)
    assert torch.equal(got, want) and moe.device_error(ws) == 0
    # a page with a key that is seen is still asked for
    b, first = max(enumerate(behind(batch, window)), key=lambda x: x[1])
    table[b, first // page] = -1
    moe.kv_attention(q, cache, *batch.args[:2], table, window=window, workspace=ws)
    assert moe.device_error(ws) == -7


@pytest.mark.parametrize("window", [1, 17, 100, 129])
@pytest.mark.parametrize("seqs", WINDOWED, ids=["one", "few", "many"])
@pytest.mark.parametrize("page,dim", [(16, 64), (64, 128), (128, 64)])
def test_what_is_behind_the_window_reaches_nobody(page, dim, seqs, window):
    """Entries of pages that hold another sequence's tokens, or nothing yet (codes and scales of any bits), and
    such codes before the first seen key of a page."""
    batch = ref.Batch(seqs, page, seed=21)
    cache = ref.filled_cache(batch, 2, dim, 21)
    q = queries(batch.T, 8, dim, 21)
    ws = space(batch, 8, cache)
    want = moe.kv_attention(q, cache, *batch.args, window=window, workspace=ws)
    ref.check_attention(q, cache, batch, want, window=window)
    for scale in (math.nan, math.inf, -1.0):
        cache.k_scale[batch.spare], cache.v_scale[batch.spare] = scale, scale
        table = batch.args[2].clone()
        for b, first in enumerate(behind(batch, window)):
            table[b, :first // page] = batch.spare[0]  # NaN codes
            p = int(batch.table[b, first // page])
            cache.k[p, :, :first % page] = 0xFF
            cache.v[p, :, :first % page] = 0x7F
        got = moe.kv_attention(q, cache, *batch.args[:2], table, window=window, workspace=ws)
        assert torch.equal(got, want) and moe.device_error(ws) == 0


@pytest.mark.parametrize("n", [1, 140])
@pytest.mark.parametrize("dim", [64, 128])
def test_scales_that_are_infinite(n, dim):
    """They count as NaN: for the rows that see the block, and for no others."""
    batch = ref.Batch([(n, 200), (n, 150)], 16, seed=9)
    cache = ref.filled_cache(batch, 2, dim, 9)
    q = queries(batch.T, 4, dim, 9)
    clean = moe.kv_attention(q, cache, *batch.args)
    page = int(batch.table[0, 12])  # tokens 192.., seen by the last 8 rows
    for scales, head in ((cache.k_scale, 0), (cache.v_scale, 1)):
        kept = scales[page].clone()
        scales[page, head] = math.inf
        got = moe.kv_attention(q, cache, *batch.args)
        hit = torch.zeros(batch.T, 4, dtype=torch.bool, device="cuda")
        hit[max(0, n - 8):n, 2 * head:2 * head + 2] = True
        assert got[hit].isnan().all() and torch.equal(got[~hit], clean[~hit])
        scales[page] = kept


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("seqs", [[(1, 130), (1, 700)], [(70, 130), (33, 400)]], ids=["one", "many"])
def test_scores_of_thousands_find_their_key(seqs, dim):
    """Each query is one key's direction, 2^60 long: that key's score is ahead by thousands, so that the
    output is its value (bf16 holds an E4M3 code times a power of two; a weight of any size cancels but for the
    2^-12 by which fp16 holds it) and the log sum its score (all products positive: 2^-16 of it for the sums,
    as much again for the query's parts and the exponent's argument)."""
    batch = ref.Batch(seqs, 32, seed=22)
    cache = ref.filled_cache(batch, 2, dim, 22)
    cache.k_scale.copy_(torch.where(cache.k_scale.isnan(), cache.k_scale, 2.0**-6))
    val = block.e4m3_values().cuda()
    g = torch.Generator().manual_seed(22)
    q = torch.zeros(batch.T, 4, dim, dtype=torch.float64, device="cuda")
    want, want_lse = torch.zeros_like(q), torch.zeros(batch.T, 4, dtype=torch.float64, device="cuda")
    scale = 2.0**-50
    for b, (n, length) in enumerate(seqs):
        pages = batch.args[2][b, : -(-length // 32)].long()
        for h in range(4):
            kv = h // 2
            k = (val[cache.k[pages, kv].long()] * cache.k_scale[pages, kv].double()[:, None, None]).flatten(0, 1)
            v = (val[cache.v[pages, kv].long()] * cache.v_scale[pages, kv].double()[:, None, None]).flatten(0, 1)
            for i in range(n):
                seen = length - n + i + 1
                j = int(torch.randint(seen, (), generator=g))
                x = k[j] * 2.0**60
                s = scale * (k[:seen] @ x)
                s[j], top = -math.inf, float(s[j])
                assert float(s.max()) < top - 4000
                r = batch.starts[b] + i
                q[r, h], want[r, h], want_lse[r, h] = x, v[j], top
    assert (q.bfloat16().double() == q).all() and (want.bfloat16().double() == want).all()
    lse = torch.empty(batch.T, 4, device="cuda")
    got = moe.kv_attention(q.bfloat16(), cache, *batch.args, scale=scale, lse=lse)
    assert (got.double() == want).all()
    assert ((lse.double() - want_lse).abs() <= 2.0**-14 * want_lse).all()


@pytest.mark.parametrize("n", [1, 100])
@pytest.mark.parametrize("dim", [64, 128])
def test_bad_pages_against_the_reference(n, dim):
    """The other keys' attention, as if the bad pages' tokens had never been there."""
    batch = ref.Batch([(n, 200), (n, 150)], 16, seed=23)
    cache = ref.filled_cache(batch, 2, dim, 23)
    q = queries(batch.T, 4, dim, 23)
    table = batch.args[2].clone()
    table[0, 2], table[0, 3] = -1, batch.n_pages
    ws = space(batch, 4, cache)
    lse = torch.empty(batch.T, 4, device="cuda")
    got = moe.kv_attention(q, cache, *batch.args[:2], table, workspace=ws, lse=lse)
    assert moe.device_error(ws) == -7
    batch.seqs[0] = (n, 200 - 32)  # 32 tokens before the first row
    whole = batch.args[2]
    shorter = whole.clone()
    shorter[0, 2:-2] = whole[0, 4:]
    batch.args = (*batch.args[:2], shorter)
    ref.check_attention(q, cache, batch, got, lse)


@pytest.mark.parametrize("seqs", [[(1, 257), (1, 1000)], [(100, 100), (37, 400)]], ids=["one", "many"])
@pytest.mark.parametrize("dim", [64, 128])
def test_value_scales_up_to_2_to_100_apart(seqs, dim):
    """A key's weight and its block's scale share one exponent.  A weight is lost where that product is 2^132
    below the row's largest, so is 2^-32 of that key's weight or less where the scales are 2^100 apart: a
    thousand such keys stay within the 2^-20 that the log sum has."""
    batch = ref.Batch(seqs, 16, seed=24)
    cache = ref.filled_cache(batch, 2, dim, 24, scales=(-64, 37))
    cache.k_scale.copy_(torch.where(cache.k_scale.isnan(), cache.k_scale, 2.0**-6))
    q = queries(batch.T, 4, dim, 24)
    lse = torch.empty(batch.T, 4, device="cuda")
    got = moe.kv_attention(q, cache, *batch.args, lse=lse)
    ref.check_attention(q, cache, batch, got, lse)
