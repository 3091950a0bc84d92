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


@pytest.mark.parametrize("max_q", [8, 99])
@pytest.mark.parametrize("cu,good", [([0, 3, 99], [(0, 0, 3)]), ([0, -4, 5], []), ([5, 3, 12], []), ([-2, 3, 5], [(1, 3, 5)]),
                                     ([0, 12, 13], [(0, 0, 12)]), ([3, 3, 2 ** 31 - 1], []),
                                     ([-2 ** 31, 0, 2], [(1, 0, 2)])])
def test_rows_around_q_and_of_refused_sequences_stay(cu, good, max_q):
    """`good`: (sequence, first row, end) of the valid ones; the rows of the others, and
    what lies around the output, are left as they were."""
    lens, T = [70, 33], 12
    q, pools, tables = build(lens, [3, 9], 4, 4, 64, torch.float16, seed=11)
    t, n, _ = dev(tables, lens, [3, 9])
    c = torch.tensor(cu, dtype=torch.int32, device=DEV)
    around = torch.full((3 * T, 4, 64), 7.0, dtype=torch.float16, device=DEV)
    out = around[T:2 * T]
    pa.paged_cross_attention(q.to(DEV), pools[0].to(DEV), pools[1].to(DEV), t, n, 0.125, max_enc_len=70, cu_q_lens=c,
                             max_q_len=max_q, out=out)
    torch.cuda.synchronize()
    assert pa.device_error() == SEQ_LEN
    left = torch.ones(3 * T, dtype=torch.bool)
    for b, lo, hi in good:
        if hi - lo <= max_q:
            check(out[lo:hi], q[lo:hi], pools, tables[b:b + 1], lens[b:b + 1], [hi - lo], 0.125)
            left[T + lo:T + hi] = False
    assert bool((around[left.to(DEV)] == 7).all())


@pytest.mark.parametrize("D", [64, 128])
def test_sequences_with_no_block_in_the_pool(D):
    """Rows of zeros, as without states; also where only the first or the last key
    tiles (of 128 states) of a chunk lie outside."""
    lens, qlens = [200, 500, 40, 700, 700, 16], [3, 30, 1, 20, 140, 9]
    q, pools, tables = build(lens, qlens, 8, 2, D, torch.float16, seed=22)
    NB = pools[0].shape[0]
    for b in (0, 1, 2, 5):
        tables[b, :] = [-1, NB, 2 ** 31 - 1, -2 ** 31][b % 4]
    tables[3, :16] = NB + 1          # the first two tiles and the last ones
    tables[4, 24:] = -7
    out = pa.paged_cross_attention(q.to(DEV), pools[0].to(DEV), pools[1].to(DEV), *dev(tables, lens, qlens)[:2],
                                   1 / math.sqrt(D), max_enc_len=700, cu_q_lens=dev(tables, lens, qlens)[2], max_q_len=140)
    torch.cuda.synchronize()
    assert pa.device_error() == BLOCK_ID
    check(out, q, pools, tables, lens, qlens, 1 / math.sqrt(D))
    at = 0
    for b, c in enumerate(qlens):
        if b in (0, 1, 2, 5):
            assert not out[at:at + c].any()
        at += c
