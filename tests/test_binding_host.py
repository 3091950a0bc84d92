"""What the wrappers hand to the library, on the CPU with a stand-in library."""
import pytest
import torch

import paged_kv_attention_decode_gb300 as pa
from tests._stand_in import StandIn, dev


@pytest.fixture
def lib(monkeypatch):
    return StandIn(monkeypatch)


@pytest.mark.parametrize("shape,dtype,elem", [
    ((6, 16, 8, 128), torch.float16, 2),       # 16-bit, token-major
    ((6, 8, 16, 128), torch.uint8, 1),         # FP8, head-major: fewer, as many and more heads than tokens
    ((6, 16, 16, 128), torch.uint8, 1),
    ((6, 40, 16, 128), torch.float8_e4m3fn, 1),
    ((6, 1, 16, 128), torch.uint8, 1),
    ((6, 5, 9 * 128), torch.uint8, 1),         # 4-bit tiles
    ((6, 3, 9 * 64), torch.uint8, 1),
])
def test_copy_blocks_passes_the_bytes_of_a_block(lib, shape, dtype, elem):
    k, v = (dev(torch.zeros(shape, dtype=torch.uint8).to(dtype)) for _ in range(2))
    pa.copy_blocks(k, v, dev(torch.zeros(2, 2, dtype=torch.int32)))
    (name, args), = lib.calls
    assert name == "pa_copy_blocks" and args[3:5] == (2, 6) and args[7] == elem
    block = 16 * args[5] * args[6] * args[7]                 # as the header defines it
    assert block == k[0].numel() * k.element_size()


@pytest.mark.parametrize("shape,dtype", [
    ((6, 8, 16), torch.float16), ((6, 2, 8, 16, 128), torch.uint8), ((6, 8, 8, 128), torch.float16),
    ((6, 3, 4, 24), torch.uint8),
])
def test_copy_blocks_refuses_other_pools(lib, shape, dtype):
    k, v = (dev(torch.zeros(shape, dtype=torch.uint8).to(dtype)) for _ in range(2))
    with pytest.raises(pa.PagedAttnError):
        pa.copy_blocks(k, v, dev(torch.zeros(2, 2, dtype=torch.int32)))
    assert not lib.calls
