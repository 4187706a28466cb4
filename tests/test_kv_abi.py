"""Refusals of the paged cache's calls, on the host: nothing is launched, no pointer is read."""
import ctypes

import pytest
import torch

import w8a8_quantised_moe_gb300 as moe
from w8a8_quantised_moe_gb300 import _lib
from w8a8_quantised_moe_gb300 import build as lib_build

OK, INVALID, SHAPE, WS_SMALL, CUDA = 0, -1, -2, -3, -4
FAKE = 1 << 20  # an aligned, never dereferenced address
CACHE = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, n_pages=10, heads=2, page=64, dim=128,
             page_stride=2 * 64 * 128, scale_stride=2)
BATCH = dict(q_start=FAKE, lengths=FAKE, page_table=FAKE, B=3, T=5, max_pages=4, table_stride=4)


@pytest.fixture(scope="module")
def lib():
    lib_build.build()
    return _lib.load()


def structs(given):
    c = _lib.KvCacheT(**{n: given.pop(n, v) for n, v in CACHE.items()})
    b = _lib.KvBatchT(**{n: given.pop(n, v) for n, v in BATCH.items()})
    return c, b


def append(lib, **given):
    c, b = structs(given)
    a = dict(key=FAKE, k_stride=256, value=FAKE, v_stride=256, q=FAKE, q_stride=512, q_heads=4, rope=FAKE,
             rope_rows=100, rope_dim=64, interleaved=0, q_out=FAKE, ws=FAKE, ws_bytes=256)
    a.update(given)
    return lib.moe_w8a8_kv_append(ctypes.addressof(c), ctypes.addressof(b), *a.values(), None)


def attend(lib, short=0, **given):
    c, b = structs(given)
    a = dict(q=FAKE, q_stride=512, q_heads=4, scale=0.1, window=0, out=2 * FAKE, lse=None, ws=FAKE)
    a.update(given)
    need = lib.moe_w8a8_kv_attention_workspace_size(b.B, b.T, a["q_heads"], c.heads, c.dim) or 1 << 40
    return lib.moe_w8a8_kv_attention(ctypes.addressof(c), ctypes.addressof(b), *a.values(), need - short, None)


BAD_SHAPES = [dict(heads=0), dict(heads=257), dict(dim=96), dict(dim=256), dict(page=8), dict(page=48), dict(page=256),
              dict(n_pages=-1), dict(n_pages=1 << 31), dict(page_stride=2 * 64 * 128 - 16),
              dict(page_stride=2 * 64 * 128 + 8), dict(scale_stride=1), dict(B=-1), dict(T=-1), dict(B=(1 << 20) + 1),
              dict(T=(1 << 20) + 1), dict(max_pages=-1), dict(max_pages=1 << 25, table_stride=1 << 25),
              dict(table_stride=3)]
POINTERS_16 = ["k", "v", "q", "ws"]
POINTERS_4 = ["k_scale", "v_scale", "q_start", "lengths", "page_table"]


@pytest.mark.parametrize("call", [append, attend])
def test_shapes(lib, call):
    for bad in BAD_SHAPES + [dict(q_heads=1025), dict(q_stride=504), dict(q_stride=516)]:
        assert call(lib, **bad) == SHAPE, bad
    assert call(lib, B=0, q=None) == OK and call(lib, T=0, q_start=None) == OK


@pytest.mark.parametrize("call", [append, attend])
def test_pointers(lib, call, monkeypatch):
    for name in POINTERS_16 + (["key", "value", "rope", "q_out"] if call is append else ["out"]):
        if not (call is append and name in ("q", "rope")):
            assert call(lib, **{name: None}) == INVALID, name
        assert call(lib, **{name: FAKE + 8}) == INVALID, name
    for name in POINTERS_4:
        assert call(lib, **{name: None}) == INVALID and call(lib, **{name: FAKE + 2}) == INVALID, name
    null = [None, None] + [0] * 12 + [FAKE, 256, None]
    assert lib.moe_w8a8_kv_append(*null) == INVALID
    monkeypatch.setenv("MOE_INJECT", "bad_ptr")
    assert call(lib) == INVALID
    monkeypatch.setenv("MOE_INJECT", "ws_short")
    assert call(lib) == WS_SMALL
    monkeypatch.setenv("MOE_INJECT", "launch_fail")
    assert call(lib) == CUDA


def test_append_only(lib):
    for bad in (dict(k_stride=248), dict(v_stride=260), dict(rope_dim=136), dict(rope_dim=24), dict(rope_dim=144),
                dict(rope_rows=-1), dict(q_heads=0)):
        assert append(lib, **bad) == SHAPE, bad
    assert append(lib, rope=None) == INVALID and append(lib, rope_dim=0) == INVALID
    assert append(lib, ws_bytes=255) == WS_SMALL
    assert append(lib, q_stride=520) == INVALID  # in place, but not contiguous


def test_attention_only(lib):
    for bad in (dict(q_heads=1), dict(q_heads=5), dict(q_heads=0)):
        assert attend(lib, **bad) == SHAPE, bad
    for bad in (dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
                dict(window=-1), dict(lse=FAKE + 2), dict(ws=FAKE + 128), dict(out=FAKE)):
        assert attend(lib, **bad) == INVALID, bad
    assert attend(lib, short=1) == WS_SMALL


def test_a_workspace_for_a_larger_batch_serves_smaller_ones(lib):
    size = lib.moe_w8a8_kv_attention_workspace_size
    for Hq, Hkv, D in ((1, 1, 64), (32, 8, 128), (56, 8, 128), (128, 1, 128), (40, 40, 64)):
        for B in (0, 1, 7, 64, 4096):
            need = [size(B, T, Hq, Hkv, D) for T in [*range(0, 3000), 1 << 14, 1 << 20]]
            assert need[0] > 0 and all(a <= b for a, b in zip(need, need[1:]))
        for T in (1, 64, 1000, 8192):
            need = [size(B, T, Hq, Hkv, D) for B in [*range(0, 300), 1 << 20]]
            assert all(a <= b for a, b in zip(need, need[1:]))
    for bad in ((1, 1, 3, 2, 64), (1, 1, 2, 0, 64), (1, 1, 2, 2, 80), (-1, 1, 2, 2, 64), (1, -1, 2, 2, 64),
                (1, 1 << 20, 1024, 1, 128 * 3)):
        assert size(*bad) == 0


def cpu_cache(n=4, heads=2, page=16, dim=64):
    return [torch.zeros(n, heads, page, dim, dtype=torch.uint8) for _ in range(2)], [torch.zeros(n, heads)] * 2


def test_python_refusals():
    codes, scales = cpu_cache()
    with pytest.raises(ValueError, match="k: expected cuda"):
        moe.KVCache(*codes, *scales)
    with pytest.raises(ValueError, match="4 dimensions"):
        moe.KVCache(codes[0][0], codes[1], *scales)
    with pytest.raises(moe.MoeError):
        moe.kv_attention_workspace_size(1, 1, 3, 2, 64)

    class Handle:
        heads, page, dim, device, _index = 2, 16, 64, "cuda:0", 0
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    ints = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="k: expected torch.bfloat16"):
        moe.kv_append(Handle, x, x, ints, ints[:2], ints[:2, None])
    with pytest.raises(ValueError, match="q: expected torch.bfloat16"):
        moe.kv_attention(x, Handle, ints, ints[:2], ints[:2, None])
    with pytest.raises(ValueError, match="lengths: expected contiguous torch.int32"):
        moe._kv_batch(ints, ints[:2], ints[:2, None], 4, Handle)
    Handle._index = -1  # the host's tensors pass, but for what is wrong with each
    with pytest.raises(ValueError, match="v: expected torch.bfloat16"):
        moe.kv_append(Handle, x, x[:, :1], ints, ints[:2], ints[:2, None])
    with pytest.raises(ValueError, match="q_start: expected"):
        moe.kv_append(Handle, x, x, ints[:2], ints[:2], ints[:2, None])
    with pytest.raises(ValueError, match="page_table: expected"):
        moe.kv_append(Handle, x, x, ints, ints[:2], ints[:1, None])
    with pytest.raises(ValueError, match="rope: expected"):
        moe.kv_append(Handle, x, x, ints, ints[:2], ints[:2, None], rope=torch.zeros(4, 4, dtype=torch.float64))
    with pytest.raises(ValueError, match="q_out: expected"):
        moe.kv_append(Handle, x, x, ints, ints[:2], ints[:2, None], q=x, q_out=x[:2])
    with pytest.raises(ValueError, match="lse: expected"):
        moe.kv_attention(x, Handle, ints, ints[:2], ints[:2, None], lse=torch.zeros(4, 3))
