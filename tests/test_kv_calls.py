"""The paged cache's Python calls without a GPU: what they allocate belongs to the stream
they are given, and workspaces are device memory (the library and the streams are stand-ins)."""
import os
import re

import pytest
import torch

import test_stream_allocations as calls
import w8a8_quantised_moe_gb300 as moe
from w8a8_quantised_moe_gb300 import _lib
from w8a8_quantised_moe_gb300 import build

allocations = calls.allocations  # the fixture


class Cache:
    heads, page, dim, device, _at, _status_at = 2, 16, 64, "cpu", 0, 0


ROWS = torch.ones(3, 2, 64, dtype=torch.bfloat16)
INTS = torch.zeros(3, dtype=torch.int32)
BATCH = (INTS, INTS[:2], INTS[:2, None])


@pytest.fixture
def stand_ins(monkeypatch):
    monkeypatch.setattr(_lib, "load", lambda: calls.FakeLibrary())
    monkeypatch.setattr(moe, "_rows_fit", lambda *a: True)
    monkeypatch.setattr(moe, "_fits_cache", lambda *a: True)
    monkeypatch.setattr(moe, "_raw_stream", lambda stream, t: 0)
    monkeypatch.setattr(moe, "_kv_batch", lambda *a: _lib.KvBatchT(0, 0, 0, 2, 3, 1, 1))


def append(**kw):
    return moe.kv_append(Cache, ROWS, ROWS, *BATCH, q=ROWS, **kw)


def attention(**kw):
    return moe.kv_attention(ROWS, Cache, *BATCH, **kw)


@pytest.mark.parametrize("call", [append, attention])
def test_a_call_allocates_on_its_stream(call, stand_ins, allocations):
    call()
    plain = [n for n, _ in allocations]
    assert plain and all(s is None for _, s in allocations)
    del allocations[:]
    s = calls.FakeStream()
    call(stream=s)
    assert [n for n, _ in allocations] == plain and all(under is s for _, under in allocations)


def test_a_call_with_its_buffers_given_allocates_nothing(stand_ins, allocations):
    s, out, ws = calls.FakeStream(), ROWS.clone(), torch.ones(4096, dtype=torch.uint8)
    assert append(stream=s, q_out=out) is out
    assert attention(stream=s, out=out, workspace=ws) is out
    assert moe.kv_append(Cache, ROWS, ROWS, *BATCH, stream=s) is None
    assert allocations == []


def test_a_workspace_in_host_memory_is_refused(stand_ins):
    with pytest.raises(ValueError, match="workspace: expected a contiguous cuda tensor"):
        attention(workspace=torch.zeros(4096, dtype=torch.uint8))


def test_the_trigger_follows_the_allocation_of_tensor_memory():
    """As for the other kernels with tensor memory: the next kernel on the stream may start only
    once this one holds its columns."""
    with open(os.path.join(build.CSRC, "kv_attend.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    alloc = re.search(r"if \(warp == kTcProducts0\) \{\s*tmem_alloc\(", text)
    assert alloc and len(re.findall(r"\btmem_alloc\(", text)) == 1
    triggers = [m.start() for m in re.finditer(r"pdl_trigger\(\);", text)]
    assert len(triggers) == 1 and triggers[0] > alloc.end()
    assert text[:triggers[0]].rstrip().endswith("if (warp == kTcProducts0)")
