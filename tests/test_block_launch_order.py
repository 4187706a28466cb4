"""A block-scaled kernel lets the next kernel on the stream start only once it holds its
tensor memory: the next one, started on the same SM, could otherwise take the columns and
wait for this kernel's end while this kernel waits for the columns, both without a limit.
Read from the sources (CPU)."""
import os
import re

import pytest

from w8a8_quantised_moe_gb300 import build

KERNELS = ["gemm_block.cu", "gemm_block_few.cu", "linear_block_few.cu"]


@pytest.mark.parametrize("name", KERNELS)
def test_the_trigger_follows_the_allocation(name):
    with open(os.path.join(build.CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    alloc = re.search(r"if \(warp == (\d+)\) \{\s*tmem_alloc\(", text)
    assert alloc and len(re.findall(r"\btmem_alloc\(", text)) == 1
    barrier = text.index("__syncthreads();", alloc.end())  # the one that publishes the address
    triggers = [m.start() for m in re.finditer(r"pdl_trigger\(\);", text)]
    assert triggers
    for at in triggers:
        by_the_allocating_warp = text[:at].rstrip().endswith(f"if (warp == {alloc.group(1)})")
        assert at > barrier or (at > alloc.end() and by_the_allocating_warp), text[at - 80:at + 15]


def test_a_cta_with_all_columns_leaves_no_shared_memory_for_another():
    """The linear layer's form for 65 to 128 rows holds all 512 columns: with a second cluster kernel on
    its SM (from another stream) each could hold an SM that a CTA of the other's cluster waits for."""
    with open(os.path.join(build.CSRC, "linear_block_few.cu")) as f:
        text = f.read()
    assert re.search(r"if \(ntok \* kLfNS == 512 && L\.total < kLfMaxSmem\) L\.total = kLfMaxSmem;", text)
