"""Appending to the paged 8-bit cache: the codes and scales are exactly the definition's."""
import pytest
import torch

import kv_reference as ref
import w8a8_quantised_moe_gb300 as moe

pytestmark = pytest.mark.gpu


def rows(T, heads, dim, seed, wide=0, size=1.0):
    """bf16 [T, heads, dim], part of rows `wide` channels wider."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = size * torch.randn(T, heads * dim + wide, generator=g, device="cuda")
    x[:, ::17] *= 20
    return x.bfloat16()[:, wide // 2:wide // 2 + heads * dim].unflatten(1, (heads, dim))


def run(seqs, page, dim, heads=2, q_heads=6, rope_dim=None, interleaved=False, seed=0, wide=0, extra_rows=0,
        positions=None):
    batch = ref.Batch(seqs, page, seed=seed, extra_rows=extra_rows)
    cache = ref.filled_cache(batch, heads, dim, seed)
    want = ref.Stored(cache)
    k, v, q = (rows(batch.T, h, dim, seed + i, wide) for i, h in enumerate((heads, heads, q_heads)))
    rope_dim = dim if rope_dim is None else rope_dim
    rope = ref.rope_table(positions or max(length for _, length in seqs), rope_dim) if rope_dim else None
    got = moe.kv_append(cache, k, v, *batch.args, q=q, rope=rope, interleaved=interleaved)
    want.append(k, v, batch, rope, interleaved)
    want.check(cache)
    ref.check_queries(q, got, batch, rope, interleaved)
    return batch, cache, got


ONE = [(1, 1), (1, 2), (1, 16), (1, 17), (1, 64), (1, 65), (1, 128), (1, 129), (1, 300)]
MANY = [(5, 5), (37, 100), (0, 50), (130, 257), (1, 40), (16, 16), (64, 128)]


@pytest.mark.parametrize("seqs", [ONE, MANY, [(700, 700)], [(1, 5000)]], ids=["one", "many", "prompt", "far"])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dim", [64, 128])
def test_append(seqs, page, dim):
    _, cache, _ = run(seqs, page, dim)
    assert moe.device_error(cache.status) == 0


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rope_dim", [(64, 0), (64, 16), (64, 48), (128, 16), (128, 64), (128, 112), (128, 128)])
def test_turned_channels(dim, rope_dim, interleaved):
    run(MANY, 16, dim, rope_dim=rope_dim, interleaved=interleaved, heads=3, seed=1)


@pytest.mark.parametrize("heads,q_heads", [(1, 1), (5, 15), (8, 56), (4, 128), (9, 9), (1, 1024)])
def test_heads(heads, q_heads):
    run([(3, 20), (1, 33), (40, 40)], 32, 64, heads, q_heads, seed=2)
    run([(1, 20), (1, 33)], 32, 64, heads, q_heads, seed=2)


def test_parts_of_wider_rows():
    run(MANY, 32, 128, wide=48, seed=3)
    run(ONE, 32, 128, wide=272, seed=3)


@pytest.mark.parametrize("count,most", [(700, 4), (2500, 4), (1100, 60)])
def test_many_sequences(count, most):
    g = torch.Generator().manual_seed(4)
    run([(int(torch.randint(0, most, (), generator=g)), int(torch.randint(4, 70, (), generator=g))) for _ in range(count)],
        16, 64, 1, 2, rope_dim=16, seed=4)


def test_rows_behind_the_last_sequence_are_left_alone():
    batch = ref.Batch([(2, 9), (1, 1)], 16, extra_rows=4)
    cache = ref.filled_cache(batch, 2, 64)
    k, v, q = (rows(batch.T, h, 64, i) for i, h in enumerate((2, 2, 4)))
    k[3:], v[3:], q[3:] = float("nan"), float("nan"), float("nan")
    want = ref.Stored(cache)
    out = torch.full((batch.T, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    got = moe.kv_append(cache, k, v, *batch.args, q=q, rope=ref.rope_table(9, 64), q_out=out)
    assert got is out and (out[3:] == 7).all()
    want.append(k, v, batch, ref.rope_table(9, 64))
    want.check(cache)


def test_a_page_filled_token_by_token():
    """Scales grow now and then; old codes are rounded again each time."""
    page, dim, heads = 32, 64, 3
    cache = moe.new_kv_cache(4, heads, dim, page)
    want = ref.Stored(cache)
    for length in range(1, 3 * page + 2):
        batch = ref.Batch([(1, length)], page, n_pages=4, seed=9, extra_pages=0)
        size = 2.0 ** ((length * 7) % 23 - 11)
        k, v = rows(1, heads, dim, length, size=size), rows(1, heads, dim, length + 500, size=1 / size)
        moe.kv_append(cache, k, v, *batch.args)
        want.append(k, v, batch)
    want.check(cache)


@pytest.mark.parametrize("n", [1, 40])
def test_sizes_of_values(n):
    """Blocks of zeros, of the type's smallest and largest values, and at the border of a scale."""
    for size in (0.0, 2.0**-133, 2.0**-64, 2.0**-66, 448.0, 449.0, 446.0, 2.0**127, float(torch.finfo(torch.bfloat16).max)):
        batch = ref.Batch([(n, 50)], 32)
        cache = ref.filled_cache(batch, 2, 64)
        want = ref.Stored(cache)
        k = torch.full((n, 2, 64), size, device="cuda").bfloat16()
        k[:, 1, ::2] *= -1
        moe.kv_append(cache, k, k, *batch.args)
        want.append(k, k, batch)
        want.check(cache)


@pytest.mark.parametrize("n", [1, 20])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_what_is_not_finite_stays_in_its_block(n, bad):
    batch = ref.Batch([(n, 40), (n, 41)], 32)
    cache = ref.filled_cache(batch, 2, 64)
    want = ref.Stored(cache)
    k, v = rows(2 * n, 2, 64, 1), rows(2 * n, 2, 64, 2)
    k[n - 1, 1, 3] = v[2 * n - 1, 0, 5] = bad
    rope = ref.rope_table(41, 32)
    moe.kv_append(cache, k, v, *batch.args, rope=rope)
    want.append(k, v, batch, rope)
    want.check(cache)
    assert int(cache.k_scale.isnan().sum()) >= 1
    nan_codes = [((c[batch.table[0, 1]] & 0x7F) == 0x7F)[:, 8 - min(n, 8):8].any() for c in (cache.k, cache.v)]
    assert not any(nan_codes)
    # the page stays so until it is begun anew
    later = ref.Batch([(1, 41), (1, 42)], 32)
    later.table, later.args = batch.table, (later.args[0], later.args[1], batch.args[2])
    moe.kv_append(cache, k[:2], v[:2], *later.args, rope=ref.rope_table(42, 32))
    assert cache.k_scale[batch.table[0, 1], 1].isnan()


def test_shorter_than_their_new_tokens():
    run([(5, 3), (4, 0), (3, 20)], 16, 64, seed=5)


@pytest.mark.parametrize("n", [1, 30])
def test_positions_outside_the_table(n):
    batch, cache, _ = run([(n, 40), (n, 61), (n, 90)], 32, 64, positions=60, seed=6)
    with pytest.raises(moe.MoeError, match="MOE_ERR_DEVICE"):
        moe._lib.check(moe.device_error(cache.status), "kv_append")


@pytest.mark.parametrize("n", [1, 30])
@pytest.mark.parametrize("bad", [-1, 1 << 30, "n_pages"])
def test_bad_pages(n, bad):
    batch = ref.Batch([(n, 40), (n, 61), (n, 90)], 32)
    bad = batch.n_pages if bad == "n_pages" else bad
    batch.table[1, 1] = bad
    batch.table[1, 0] = bad
    batch.args = (*batch.args[:2], batch.table.cuda())
    cache = ref.filled_cache(ref.Batch([(0, 0)] * 3, 32, n_pages=batch.n_pages), 2, 64)
    want = ref.Stored(cache)
    k, v, q = (rows(batch.T, 2, 64, i) for i in range(3))
    got = moe.kv_append(cache, k, v, *batch.args, q=q)
    want.append(k, v, batch)
    want.check(cache)
    assert torch.equal(got, q)
    assert moe.device_error(cache.status) == -7 and moe.device_error(cache.status) == 0


@pytest.mark.parametrize("n", [1, 30])
def test_pools_with_other_strides(n):
    """Keys and values of a page next to each other, in a pool of two layers."""
    batch = ref.Batch([(n, 40), (n, 61)], 32)
    pool = torch.zeros(batch.n_pages, 2, 2, 3, 32, 64, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(batch.n_pages, 2, 2, 3, device="cuda")
    cache = moe.KVCache(pool[:, 1, 0], pool[:, 1, 1], scales[:, 1, 0], scales[:, 1, 1])
    want = ref.Stored(cache)
    k, v = rows(batch.T, 3, 64, 1), rows(batch.T, 3, 64, 2)
    table = torch.zeros(2, 9, dtype=torch.int32, device="cuda")
    table[:, :batch.table.shape[1]] = batch.args[2]
    moe.kv_append(cache, k, v, *batch.args[:2], table[:, :batch.table.shape[1]])
    want.append(k, v, batch)
    want.check(cache)
    assert not pool[:, 0].any() and not scales[:, 0].any()


def test_queries_in_place_and_nothing_to_do():
    batch = ref.Batch([(3, 9)], 16)
    cache = ref.filled_cache(batch, 1, 64)
    k, q = rows(3, 1, 64, 1), rows(3, 4, 64, 2).contiguous()
    rope = ref.rope_table(9, 64)
    want = moe.kv_append(cache, k, k, *batch.args, q=q, rope=rope)
    assert moe.kv_append(cache, k, k, *batch.args, q=q, rope=rope, q_out=q) is q and torch.equal(q, want)
    assert moe.kv_append(cache, k, k, *batch.args, rope=rope) is None
    none = ref.Batch([], 16)
    assert moe.kv_append(cache, k[:0], k[:0], *none.args, q=q[:0]).shape == (0, 4, 64)


def test_a_captured_call_follows_the_lengths():
    page, dim = 16, 64
    cache, eager = (moe.new_kv_cache(8, 2, dim, page) for _ in range(2))
    table = torch.tensor([[3, 1, 5], [0, 7, 2]], dtype=torch.int32, device="cuda")
    q_start = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    lengths = torch.tensor([1, 20], dtype=torch.int32, device="cuda")
    k, v, q = (rows(2, 2, dim, i) for i in range(3))
    rope, out = ref.rope_table(48, dim), torch.empty(2, 2, dim, dtype=torch.bfloat16, device="cuda")

    def call(c):
        return moe.kv_append(c, k, v, q_start, lengths, table, q=q, rope=rope, q_out=out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(eager)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(cache)
    for step in range(20):
        if step:
            lengths += 1
            for i, x in enumerate((k, v, q)):
                x.copy_(rows(2, 2, dim, 10 * step + i))
        graph.replay()
        got = out.clone()
        want = call(eager)
        assert torch.equal(got, want)
    for name in ("k", "v", "k_scale", "v_scale"):
        assert torch.equal(getattr(cache, name), getattr(eager, name)), name
