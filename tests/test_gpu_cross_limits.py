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


@pytest.mark.parametrize("max_q", [1, 5, 8, 9, 40, 10 ** 6])
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (64, 1)])
def test_rows_beyond_max_q_len(Hq, Hkv, max_q):
    """With max_q_len of 8 or less, more rows than that are flagged and not written;
    above, longer chunks are computed."""
    lens, qlens = [70, 300, 33, 500, 0, 64], [1, 150, 5, 41, 60, 8]
    q, pools, tables = build(lens, qlens, Hq, Hkv, 64, torch.float16, seed=21)
    t, n, cu = dev(tables, lens, qlens)
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device=DEV)
    pa.paged_cross_attention(q.to(DEV), pools[0].to(DEV), pools[1].to(DEV), t, n, 0.125, max_enc_len=500,
                             cu_q_lens=cu, max_q_len=max_q, out=out)
    torch.cuda.synchronize()
    assert pa.device_error() == (SEQ_LEN if max_q <= 8 else 0)
    at = 0
    for b, c in enumerate(qlens):
        rows = slice(at, at + c)
        at += c
        if c <= max_q or max_q > 8:
            check(out[rows], q[rows], pools, tables[b:b + 1], lens[b:b + 1], [c], 0.125)
        else:
            assert bool((out[rows] == 7).all())
