"""Cross attention: loose bounds, rows outside the queries, chunks longer than
max_q_len, and sequences whose blocks all lie outside the pool."""
import math

import pytest
import torch

import paged_kv_attention_decode_gb300 as pa
from tests.test_gpu_cross import DEV, build, check, dev

pytestmark = pytest.mark.gpu
SEQ_LEN, BLOCK_ID = 4, 1


@pytest.mark.parametrize("bound", [2 ** 31 - 1, 2 ** 31 - 14, 2 ** 40])
@pytest.mark.parametrize("qlens", [[3, 1, 8], [3, 40, 200]])
def test_bounds_that_say_nothing(qlens, bound):
    """The largest bounds of lengths are no bounds."""
    lens = [900, 33, 250]
    q, pools, tables = build(lens, qlens, 8, 2, 64, torch.float16, seed=20)
    t, n, cu = dev(tables, lens, qlens)
    out = pa.paged_cross_attention(q.to(DEV), pools[0].to(DEV), pools[1].to(DEV), t, n, 0.125, max_enc_len=bound,
                                   cu_q_lens=cu, max_q_len=bound)
    torch.cuda.synchronize()
    check(out, q, pools, tables, lens, qlens, 0.125)
    assert pa.device_error() == 0
