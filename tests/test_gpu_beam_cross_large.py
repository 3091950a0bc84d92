"""Cross attention and the beam calls where offsets pass 32 bits: pools of more
than 2^31 elements, logit rows more than 2^31 elements apart."""
import numpy as np
import pytest
import torch

import paged_kv_attention_decode_gb300 as pa
from tests import _beam_ref as B
from tests import test_gpu_beam as TB
from tests import test_gpu_cross as TC

pytestmark = pytest.mark.gpu
DEV = "cuda"
NB, H, D = 140_000, 8, 128            # 16 * 8 * 128 * 140,000 = 2.3e9 elements a pool


def room(nbytes):
    if torch.cuda.mem_get_info()[0] < nbytes + (4 << 30):
        pytest.skip("needs free device memory")


@pytest.mark.parametrize("qlens", [[3, 2, 4], [1, 30, 2]])
def test_cross_attention_over_a_large_pool(qlens):
    room(2 * NB * 16 * H * D * 2)
    lens = [100, 333, 17]
    q, pools, tables = TC.build(lens, qlens, H, H, D, torch.bfloat16, seed=31)
    ids = NB - 1 - 3 * np.arange(pools[0].shape[0])                # block i of the small pool lies here
    big = [torch.empty((NB, 16, H, D), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    for b, p in zip(big, pools):
        b[torch.from_numpy(ids).to(DEV)] = p.to(DEV)
    far = tables.copy()
    for s, n in enumerate(lens):
        u = -(-n // 16)
        far[s, :u] = ids[tables[s, :u]]
    t, n, cu = TC.dev(far, lens, qlens)
    out = pa.paged_cross_attention(q.to(DEV), *big, t, n, 0.09, max_enc_len=333, cu_q_lens=cu, max_q_len=max(qlens))
    torch.cuda.synchronize()
    TC.check(out, q, pools, tables, lens, qlens, 0.09)
    assert pa.device_error() == 0


def test_reorder_in_a_large_pool():
    room(2 * NB * 16 * H * D * 2)
    lens, W = [45, 7, 31], 6
    tables, parents, small = TB.beams(lens, W, 1, seed=32)
    far = (NB - 1 - 2 * tables).astype(np.int32)
    (k,), (v,) = TB.pools_of("f16", small, 1, H, D, seed=32)
    ids = torch.from_numpy(NB - 1 - 2 * np.arange(small)).to(DEV)
    big = [torch.empty((NB, 16, H, D), dtype=torch.float16, device=DEV) for _ in range(2)]
    for b, p in zip(big, (k, v)):
        b[ids] = p.to(DEV)
    got = TB.reorder(far, lens, parents, [big[0]], [big[1]])
    new, copies = B.reorder(tables, lens, parents)
    assert copies and np.array_equal(got, NB - 1 - 2 * new)
    for b, p in zip(big, (k, v)):
        assert torch.equal(TB.bytes_of(b[ids]), TB.bytes_of(TB.expect(p, copies, "f16")))
    assert pa.device_error() == 0


@pytest.mark.parametrize("V", [5001, 300_000])
def test_logit_rows_far_apart(V):
    apart = 2 ** 31 + 8
    room(2 * (2 * apart + V))
    buf = torch.empty(2 * apart + V, dtype=torch.float16, device=DEV)
    rows = buf.as_strided((3, V), (apart, 1))
    x, scores = TB.make(1, 3, V, torch.float16, seed=V)
    rows.copy_(x[0].to(DEV))
    TB.check(TB.run(rows, scores, 6), x, scores, 6)
