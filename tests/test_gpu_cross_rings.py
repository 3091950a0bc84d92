"""Cross attention over long sequences with blocks outside the pool: steps of two
blocks that hold one only, in the middle of a warp's work, so that ring slots
whose rows were cleared are filled again."""
import math

import numpy as np
import pytest
import torch

import paged_kv_attention_decode_gb300 as pa
from tests import _beam_ref as B
from tests import _ref64 as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
BLOCK_ID = 1


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows", [1, 5])
@pytest.mark.parametrize("seqs", [1, 13, 31])   # split over clusters; one CTA of 8 warps an item; of 4 warps
def test_slots_of_cleared_rows_are_filled_again(seqs, rows, D):
    rng = np.random.default_rng(seqs + rows + D)
    NB, H, G, blocks = 90, 5, 2, 1601 if seqs == 1 else 901
    lens = [blocks * 16 - int(x) for x in rng.integers(0, 40, seqs)]
    pools = [torch.from_numpy((rng.standard_normal((NB, 16, H, D)) + c).astype(np.float32)).half() for c in (0, 1)]
    q = torch.from_numpy((rng.standard_normal((seqs * rows, H * G, D)) / 4).astype(np.float32)).half()
    tables = rng.integers(0, NB, (seqs, blocks)).astype(np.int32)
    # every other block, or one of a few, outside the pool: single blocks and whole steps
    bad = rng.random((seqs, blocks)) < rng.choice([0.1, 0.5, 0.8], (seqs, 1))
    tables[bad] = rng.choice(np.array([-1, NB, NB + 3, -2 ** 31, 2 ** 31 - 1], np.int32), int(bad.sum()))
    scale = 1 / math.sqrt(D)
    args = (q.to(DEV), pools[0].to(DEV), pools[1].to(DEV), torch.from_numpy(tables).to(DEV),
            torch.tensor(lens, dtype=torch.int32, device=DEV), scale)
    out = pa.paged_cross_attention(*args, max_enc_len=max(lens))
    torch.cuda.synchronize()
    assert pa.device_error() == BLOCK_ID
    kv = [p.double().numpy() for p in pools]
    ref, A, smax, cnt = B.cross_attention(q.double().numpy(), *kv, tables, lens, [rows] * seqs, scale)
    tol = R.bound(ref, A, smax, cnt, float(np.abs(kv[1]).max()), q.dtype, q.dtype)
    assert np.max(np.abs(out.double().cpu().numpy() - ref) / tol) <= 1
    for _ in range(5):
        assert torch.equal(pa.paged_cross_attention(*args, max_enc_len=max(lens)), out)
    torch.cuda.synchronize()
    assert pa.device_error() == BLOCK_ID
