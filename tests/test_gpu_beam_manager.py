"""The block manager under a beam request on the device: copies on write, and
reordering in place."""
import numpy as np
import pytest
import torch

import paged_kv_attention_decode_gb300 as pa
from tests import _beam_manager as M

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("prefix_caching", [False, True])
@pytest.mark.parametrize("n0,W", [(1, 2), (21, 4), (47, 8)])
def test_every_row_keeps_its_history(n0, W, prefix_caching):
    max_blocks, steps = 8, 60
    k = torch.full((1 + W * max_blocks, 16, 2, 64), -9, dtype=torch.float16, device=DEV)
    v = k.clone()

    def copy(src, dst):
        pa.copy_blocks(k, v, torch.tensor([[src, dst]], dtype=torch.int32, device=DEV))

    def write(blocks, slot, tokens):
        slots = torch.tensor([int(b) * 16 + slot for b in blocks], device=DEV)
        x = torch.tensor(tokens, device=DEV).half()[:, None, None].expand(-1, 2, 64).contiguous()
        pa.paged_kv_write(x, -x, k, v, slots)

    def reorder(tables, n, parents):
        t = torch.from_numpy(tables).to(DEV)
        pa.beam_reorder(t, torch.full((W,), n, dtype=torch.int32, device=DEV),
                        torch.tensor(parents[None], dtype=torch.int32, device=DEV), k, v)
        return t.cpu().numpy()

    tables, n, hist = M.search(n0, W, steps, n0 + W, prefix_caching, copy, write, reorder, max_blocks)
    assert pa.device_error() == 0
    i = np.arange(n)
    for w in range(W):
        for pool, sign in ((k, 1), (v, -1)):
            got = pool[torch.from_numpy(tables[w, i // 16].astype(np.int64)).to(DEV), torch.from_numpy(i % 16).to(DEV)].cpu()
            assert torch.equal(got, (sign * torch.tensor(hist[w])).half()[:, None, None].expand(-1, 2, 64))
