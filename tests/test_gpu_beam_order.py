"""Beam selection: the order of candidates, and scores at the ends of fp32's range."""
import math

import numpy as np
import pytest
import torch

import paged_kv_attention_decode_gb300 as pa
from tests import _beam_ref as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def select(x, scores, k, **kw):
    """x [S, W, V]; the results as numpy arrays."""
    S, W, V = x.shape
    got = pa.beam_select(x.to(DEV).view(S * W, V), torch.from_numpy(np.asarray(scores, np.float32)).to(DEV), k, **kw)
    torch.cuda.synchronize()
    return [t.cpu().numpy() for t in got]


@pytest.mark.parametrize("S", [1, 200])              # one launch, and two
@pytest.mark.parametrize("V", [40, 5000])            # few logits, and many
@pytest.mark.parametrize("dn", ["bf16", "f32"])
def test_scores_in_the_range_whose_log_probability_is_below_it(dn, V, S):
    """score + (x - largest) lies within fp32's range where x - largest does not."""
    W, k, big = 3, 7, 2.0 ** 127
    x = torch.full((S, W, V), -math.inf)
    x[:, 0, 5] = big
    x[:, 0, 7], x[:, 0, 11], x[:, 0, 13] = -1.5 * big, -1.25 * big, -1.75 * big   # 2.25 to 2.75 below the largest
    x[:, 1, 3], x[:, 1, 9] = 0.0, -0.5 * big
    x[:, 2, 0], x[:, 2, 1] = big, -1.5 * big
    scores = np.tile(np.array([1.875 * big, 0.0, -0.5 * big], np.float32), (S, 1))
    sc, par, tok = select(x.to(DT[dn]), scores, k)
    want = [(1.875, 0, 5), (0.0, 1, 3), (-0.375, 0, 11), (-0.5, 1, 9), (-0.5, 2, 0), (-0.625, 0, 7), (-0.875, 0, 13)]
    assert sc.tolist() == [[w[0] * big for w in want]] * S
    assert par.tolist() == [[w[1] for w in want]] * S and tok.tolist() == [[w[2] for w in want]] * S
    ref = B.select(x.to(DT[dn]).double().numpy()[:1], scores[:1], k)
    assert np.array_equal(ref[0][0], sc[0]) and ref[1][0].tolist() == par[0].tolist() and ref[2][0].tolist() == tok[0].tolist()
