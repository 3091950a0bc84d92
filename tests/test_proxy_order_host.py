"""Shared memory that a kernel writes with ordinary stores and a later TMA copy
fills again needs a proxy fence between the two, in every thread that stored:
a barrier between threads alone does not order the two kinds of access."""
import os
import re

import pytest

from paged_kv_attention_decode_gb300 import _binding

CSRC = os.path.join(os.path.dirname(_binding.__file__), "csrc")


def code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", ["pa_cross.cu", "pa_decode.cu", "pa_prefill_tc.cu"])
def test_kernels_that_clear_rows_of_a_ring_fence_the_stores(name):
    text = code(name)
    assert "tma_load_4d" in text and "fence_proxy_async_smem();" in text


def test_cleared_rows_of_the_cross_attention_ring():
    """The rows behind a step's states are cleared by all lanes: each fences its
    stores, before the warp meets and lane 0 may ask for the slot's next tiles."""
    text = code("pa_cross.cu")
    stores = [m.end() for m in re.finditer(r"z\[i\] = make_uint4\(0, 0, 0, 0\);", text)]
    assert len(stores) == 1
    behind = text[stores[0]:]
    fence, meet = behind.find("fence_proxy_async_smem();"), behind.find("__syncwarp();")
    assert 0 <= fence < meet
    # a slot is refilled only behind a meeting of the warp
    loop = re.search(r"while \(done < issued\) \{(.*?)\n    \}", text, re.S).group(1)
    assert loop.find("st.step(") < loop.find("__syncwarp();") < loop.find("fetch();")
