"""The 4-bit decode's merge of many partitions, held to a bound that a lost or
doubled partition exceeds (checked in test_fp4_merge_host.py)."""
import numpy as np
import pytest
import torch

import paged_kv_attention_decode_gb300 as pa
from tests._fp4_merge import CASES, KS, VS, Case

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("name", CASES)
def test_every_partition_counts_once(name):
    c = Case(**CASES[name])
    q, k, v = (x.to(DEV) for x in (c.q, *map(torch.from_numpy, c.pools)))
    bt = torch.from_numpy(c.tables).to(DEV)
    sl = torch.tensor(c.lens, dtype=torch.int32, device=DEV)
    out = pa.paged_attention_decode_fp4(q, k, v, bt, sl, c.scale, KS, VS, max(c.lens), partition_size=c.part)
    torch.cuda.synchronize()
    got = out.double().cpu().numpy()
    assert np.all(np.isfinite(got))
    for b in [0, 1, *range(2, len(c.lens), 97)]:
        worst = np.max(np.abs(got[b] - c.result(b)) / c.bound(b))
        assert worst <= 1, (b, worst)
    assert pa.device_error() == 0
