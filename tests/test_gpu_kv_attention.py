"""Attention over the paged 8-bit cache against its plain 64-bit form."""
import pytest
import torch

import kv_reference as ref
import w8a8_quantised_moe_gb300 as moe

pytestmark = pytest.mark.gpu


def queries(T, q_heads, dim, seed=0, size=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (size * torch.randn(T, q_heads, dim, generator=g, device="cuda")).bfloat16()


def run(seqs, page, dim, heads=2, q_heads=4, window=0, seed=0, size=1.0, scale=None, extra_rows=0, **filled):
    batch = ref.Batch(seqs, page, seed=seed, extra_rows=extra_rows)
    cache = ref.filled_cache(batch, heads, dim, seed, **filled)
    q = queries(batch.T, q_heads, dim, seed, size)
    lse = torch.full((batch.T, q_heads), 5.0, device="cuda")
    ws = moe.new_workspace(moe.kv_attention_workspace_size(len(seqs), batch.T, q_heads, heads, dim))
    got = moe.kv_attention(q, cache, *batch.args, scale=scale, window=window, lse=lse, workspace=ws)
    assert moe.device_error(ws) == 0
    ref.check_attention(q, cache, batch, got, lse, scale, window)
    assert (lse[batch.starts[-1]:] == 5).all()
    return batch, cache, q, got, lse


LENGTHS = [1, 2, 15, 16, 17, 31, 63, 64, 65, 127, 128, 129, 255, 257, 1000]
ONE = [(1, n) for n in LENGTHS]
FEW = [(1, 70), (2, 2), (3, 64), (0, 10), (5, 200), (4, 1001), (7, 7)]
MANY = [(100, 100), (1, 300), (37, 400), (0, 9), (129, 129), (64, 1000), (256, 256), (3, 3)]


@pytest.mark.parametrize("seqs", [ONE, FEW, MANY, [(1, 3000)], [(300, 300)], [(513, 700)]],
                         ids=["one", "few", "many", "long", "prompt", "chunk"])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dim", [64, 128])
def test_attention(seqs, page, dim):
    run(seqs, page, dim)


@pytest.mark.parametrize("heads,q_heads", [(1, 1), (3, 3), (1, 3), (2, 14), (5, 15), (1, 16), (1, 17), (2, 80), (1, 128),
                                           (8, 8), (1, 300)])
@pytest.mark.parametrize("seqs", [[(1, 130), (1, 5), (1, 64)], [(6, 130), (3, 200)], [(70, 130), (1, 99), (40, 40)]],
                         ids=["one", "few", "many"])
def test_heads(heads, q_heads, seqs):
    run(seqs, 32, 64, heads, q_heads, seed=1)


@pytest.mark.parametrize("window", [1, 2, 15, 64, 100, 129, 5000, 1 << 40])
@pytest.mark.parametrize("seqs", [ONE, FEW, MANY], ids=["one", "few", "many"])
def test_window(seqs, window):
    run(seqs, 16, 64, window=window, seed=2)
    run(seqs, 64, 128, window=window, seed=2)


def test_long():
    """Parts of a sequence on every CTA, and offsets beyond 2^32 bytes in the cache."""
    run([(1, 60000), (1, 1), (1, 9999)], 64, 128, heads=1, q_heads=5, seed=3)
    run([(20, 30000), (1, 11)], 128, 128, heads=1, q_heads=8, seed=3)


@pytest.mark.parametrize("n", [1, 300])
def test_offsets_beyond_32_bits(n):
    """The last pages of a pool of 5 GB; the rest of it is not touched."""
    page, heads, dim = 128, 8, 128
    n_pages = 5 * (1 << 30) // (heads * page * dim)
    codes = [torch.empty(n_pages, heads, page, dim, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.empty(n_pages, heads, device="cuda") for _ in range(2)]
    cache = moe.KVCache(*codes, *scales)
    length = 400
    batch = ref.Batch([(n, length)], page, n_pages=4)
    small = ref.filled_cache(batch, heads, dim)
    for name in ("k", "v", "k_scale", "v_scale"):
        getattr(cache, name)[-4:] = getattr(small, name)
    q = queries(n, 8, dim)
    args = (*batch.args[:2], torch.where(batch.args[2] < 4, batch.args[2] + n_pages - 4, batch.args[2]))
    got = moe.kv_attention(q, cache, *args)
    ref.check_attention(q, small, batch, got)
    k, v = queries(n, heads, dim, 1), queries(n, heads, dim, 2)
    want = ref.Stored(small)
    moe.kv_append(cache, k, v, *args)
    want.append(k, v, batch)
    for name in ("k", "v", "k_scale", "v_scale"):
        getattr(small, name).copy_(getattr(cache, name)[-4:])
    want.check(small)


@pytest.mark.parametrize("size", [0.0, 2.0**-120, 2.0**-30, 30.0])
@pytest.mark.parametrize("seqs", [[(1, 130)], [(70, 130)]], ids=["one", "many"])
def test_sizes_of_queries(seqs, size):
    run(seqs, 32, 128, size=size, seed=4, spread=1.0)


def test_large_queries():
    """Scores of thousands: one key has all the weight; nothing overflows."""
    for seqs in ([(1, 130)], [(70, 130)]):
        batch, cache, q, got, lse = run(seqs, 32, 64, size=2.0**60, scale=2.0**-52, seed=5)
        assert got.isfinite().all()


@pytest.mark.parametrize("scales", [(-64, -60), (-40, 10), (60, 64)])
@pytest.mark.parametrize("seqs", [ONE[5:], MANY[:4]], ids=["one", "many"])
def test_scales_of_blocks(seqs, scales):
    """Values of blocks next to each other differ by 2^50; keys' scores are kept within bounds."""
    for dim in (64, 128):
        batch = ref.Batch(seqs, 16, seed=6)
        cache = ref.filled_cache(batch, 2, dim, 6, scales=scales)
        cache.k_scale.copy_(torch.where(cache.k_scale.isnan(), cache.k_scale, 2.0**-6))
        q = queries(batch.T, 4, dim, 6)
        lse = torch.empty(batch.T, 4, device="cuda")
        got = moe.kv_attention(q, cache, *batch.args, lse=lse)
        ref.check_attention(q, cache, batch, got, lse)


def test_scales_that_are_no_powers_of_two():
    for seqs in (ONE, MANY):
        batch = ref.Batch(seqs, 16, seed=7)
        cache = ref.filled_cache(batch, 2, 64, 7)
        for s in (cache.k_scale, cache.v_scale):
            s *= 1 + torch.rand(s.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
        q = queries(batch.T, 4, 64, 7)
        ref.check_attention(q, cache, batch, moe.kv_attention(q, cache, *batch.args))


@pytest.mark.parametrize("seqs", [[(1, 0), (1, 20), (3, 1), (2, 0), (4, 4)],
                                  [(300, 0), (1, 20), (300, 100), (2, 0), (100, 99)]], ids=["few", "many"])
def test_rows_that_see_nothing(seqs):
    batch, cache, q, got, lse = run(seqs, 16, 64, heads=1, q_heads=8, seed=8)
    blind = torch.cat([torch.arange(n) < n - length for n, length in seqs]).cuda()
    assert blind.any() and not got[blind].any() and (lse[blind] == -float("inf")).all()
    assert lse[~blind].isfinite().all()
    # whatever their queries are
    q[blind] = float("nan")
    again = moe.kv_attention(q, cache, *batch.args)
    assert torch.equal(again, got)


def test_rows_behind_the_last_sequence():
    for seqs in ([(1, 20), (1, 300)], [(200, 300)]):
        batch = ref.Batch(seqs, 16, extra_rows=5)
        cache = ref.filled_cache(batch, 2, 64)
        q = queries(batch.T, 4, 64)
        q[-5:] = float("nan")
        out = torch.full_like(q, 3.0)
        ws = moe.new_workspace(moe.kv_attention_workspace_size(len(seqs), batch.T, 4, 2, 64))
        ws[256:] = 0x7F  # of an earlier call
        assert moe.kv_attention(q, cache, *batch.args, out=out, workspace=ws) is out
        ref.check_attention(q, cache, batch, out)
        assert (out[-5:] == 3).all()


@pytest.mark.parametrize("n", [1, 140])
def test_what_is_not_finite_reaches_only_who_sees_it(n):
    seqs = [(n, 200), (n, 150)]
    batch = ref.Batch(seqs, 16, seed=9)
    cache = ref.filled_cache(batch, 2, 64, 9)
    q = queries(batch.T, 4, 64, 9)
    clean = moe.kv_attention(q, cache, *batch.args)
    # sequence 0: the block of tokens 192.. of key head 0, seen by its last 8 rows; of values of head 1
    page = int(batch.table[0, 12])
    for scales, heads in ((cache.k_scale, slice(0, 2)), (cache.v_scale, slice(2, 4))):
        kept = scales[page].clone()
        scales[page, 0 if heads.start == 0 else 1] = float("nan")
        got = moe.kv_attention(q, cache, *batch.args)
        hit = torch.zeros(batch.T, 4, dtype=torch.bool, device="cuda")
        hit[max(0, n - 8):n, heads] = True
        assert got[hit].isnan().all() and torch.equal(got[~hit], clean[~hit])
        scales[page] = kept
    # a query that is not finite: its row alone
    for bad in (float("nan"), float("inf")):
        dirty = q.clone()
        dirty[n - 1, 1, 7] = bad
        got = moe.kv_attention(dirty, cache, *batch.args)
        hit = torch.zeros(batch.T, 4, dtype=torch.bool, device="cuda")
        hit[n - 1, 1] = True
        assert got[hit].isnan().any() and torch.equal(got[~hit], clean[~hit])


@pytest.mark.parametrize("n", [1, 140])
@pytest.mark.parametrize("bad", [-1, 1 << 30, "n_pages"])
def test_bad_pages_are_not_seen(n, bad):
    """The tokens of a page that is not the cache's count as not there, and the error word says so."""
    seqs = [(n, 200), (n, 150)]
    batch = ref.Batch(seqs, 16, seed=10)
    cache = ref.filled_cache(batch, 2, 64, 10)
    q = queries(batch.T, 4, 64, 10)
    table = batch.args[2].clone()
    table[0, 2:4] = batch.n_pages if bad == "n_pages" else bad
    ws = moe.new_workspace(moe.kv_attention_workspace_size(2, batch.T, 4, 2, 64))
    got = moe.kv_attention(q, cache, *batch.args[:2], table, workspace=ws)
    assert moe.device_error(ws) == -7 and moe.device_error(ws) == 0
    # the same with a value block that is not seen: a scale of 0
    pages = batch.args[2][0, 2:4].long()
    cache.v_scale[pages] = 0.0
    want = moe.kv_attention(q, cache, *batch.args, workspace=ws)
    assert moe.device_error(ws) == 0 and torch.equal(got, want)
    rows = slice(batch.starts[1], batch.starts[2])
    ref.check_attention(q, cache, batch, got, rows=rows)


def test_lengths_beyond_the_page_table():
    for n in (1, 100):
        batch = ref.Batch([(n, 160), (n, 100)], 16, extra_pages=0)
        cache = ref.filled_cache(batch, 2, 64)
        q = queries(batch.T, 4, 64)
        got = moe.kv_attention(q, cache, batch.args[0], torch.tensor([100000, 100], dtype=torch.int32).cuda(), batch.args[2])
        ref.check_attention(q, cache, batch, got)


def test_pages_of_several_sequences():
    """A beginning that two sequences share, and one page twice in a sequence."""
    for n in (1, 60):
        batch = ref.Batch([(n, 160), (n, 170)], 16, seed=11)
        batch.table[1, :6] = batch.table[0, :6]
        batch.table[1, 7] = batch.table[1, 6]
        batch.args = (*batch.args[:2], batch.table.cuda())
        cache = ref.filled_cache(batch, 2, 128, 11)
        q = queries(batch.T, 4, 128, 11)
        ref.check_attention(q, cache, batch, moe.kv_attention(q, cache, *batch.args))


def test_strided_queries_and_pools():
    for seqs in (FEW, MANY):
        batch = ref.Batch(seqs, 32, seed=12)
        cache = ref.filled_cache(batch, 3, 64, 12)
        pool = torch.full((batch.n_pages, 2, 2, 3, 32, 64), 0x7F, dtype=torch.uint8, device="cuda")
        scales = torch.full((batch.n_pages, 5, 3), float("nan"), device="cuda")
        pool[:, 0, 1], pool[:, 1, 0], scales[:, 0], scales[:, 4] = cache.k, cache.v, cache.k_scale, cache.v_scale
        wide = moe.KVCache(pool[:, 0, 1], pool[:, 1, 0], scales[:, 0], scales[:, 4])
        rows = torch.full((batch.T, 9 * 64 + 40), float("nan"), device="cuda").bfloat16()
        q = rows[:, 16:16 + 6 * 64].unflatten(1, (6, 64))
        q.copy_(queries(batch.T, 6, 64, 12))
        want = moe.kv_attention(q.contiguous(), cache, *batch.args)
        assert torch.equal(moe.kv_attention(q, wide, *batch.args), want)
        ref.check_attention(q, cache, batch, want)


def test_many_sequences():
    g = torch.Generator().manual_seed(13)
    seqs = [(int(torch.randint(0, 3, (), generator=g)), int(torch.randint(0, 90, (), generator=g))) for _ in range(1000)]
    run(seqs, 16, 64, heads=1, q_heads=2, seed=13)


@pytest.mark.parametrize("dim", [64, 128])
def test_row_tiles_with_one_tile_before_some_with_two(dim):
    """The second tile's warps pass over row tiles of at most 128 rows; what they then read is their own step's."""
    seqs = [(33, 2345), (290, 1500), (65, 3000), (288, 2100), (301, 301)]
    batch = ref.Batch(seqs, 32, seed=18)
    cache = ref.filled_cache(batch, 8, dim, 18, scales=(-8, 0))
    q = queries(batch.T, 32, dim, 18)
    first = moe.kv_attention(q, cache, *batch.args)
    ref.check_attention(q, cache, batch, first)
    lines = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for i in range(24):
        if i % 3 == 0:
            lines.fill_(i)  # the cache from memory, not from L2
        assert torch.equal(moe.kv_attention(q, cache, *batch.args), first)


def test_no_rows():
    batch = ref.Batch([], 16)
    cache = moe.new_kv_cache(1, 2, 64, 16)
    assert moe.kv_attention(queries(0, 4, 64), cache, *batch.args).shape == (0, 4, 64)
    batch = ref.Batch([(0, 5), (0, 0)], 16)
    out = torch.full((0, 4, 64), 1.0, device="cuda").bfloat16()
    assert moe.kv_attention(out, cache, *batch.args).shape == (0, 4, 64)


@pytest.mark.parametrize("seqs", [ONE, MANY], ids=["one", "many"])
def test_the_same_bits_each_time_and_on_two_streams(seqs):
    batch = ref.Batch(seqs, 16, seed=14)
    cache = ref.filled_cache(batch, 2, 128, 14)
    qs = [queries(batch.T, 8, 128, i) for i in range(2)]
    size = moe.kv_attention_workspace_size(len(seqs), batch.T, 8, 2, 128)
    spaces = [moe.new_workspace(size) for _ in range(2)]
    want = [moe.kv_attention(q, cache, *batch.args, workspace=spaces[0]).clone() for q in qs]
    outs = [torch.empty_like(w) for w in want]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for q, ws, out, s in zip(qs, spaces, outs, streams):
            moe.kv_attention(q, cache, *batch.args, workspace=ws, out=out, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("n", [1, 200])
def test_a_captured_call_follows_the_lengths(n):
    batch = ref.Batch([(n, 500), (n, 700)], 16, seed=15)
    cache = ref.filled_cache(batch, 2, 128, 15)
    q = queries(batch.T, 8, 128)
    ws = moe.new_workspace(moe.kv_attention_workspace_size(2, batch.T, 8, 2, 128))
    other = moe.new_workspace(ws.numel())
    out = torch.empty_like(q)
    lengths = batch.args[1].clone()

    def call(out, ws):
        return moe.kv_attention(q, cache, batch.args[0], lengths, batch.args[2], out=out, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(out, ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out, ws)
    for a, b in ((500, 700), (n, n), (499, 210), (500, 650)):
        lengths.copy_(torch.tensor([a, b], dtype=torch.int32))
        q.copy_(queries(batch.T, 8, 128, a))
        graph.replay()
        got = out.clone()
        assert torch.equal(got, call(torch.empty_like(q), other))
