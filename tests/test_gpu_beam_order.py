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


@pytest.mark.parametrize("S", [1, 200])
@pytest.mark.parametrize("V", [64, 5000])
@pytest.mark.parametrize("first", [0, 1])
def test_scores_that_are_one_number_in_fp32(first, V, S):
    """Two beams whose best candidates score -1000 and -1000 - 44 e^-16 (5e-6 less, where a
    unit of fp32 is 6e-5): equal once rounded, in their order all the same."""
    W = 2
    x = torch.full((S, W, V), -60.0)
    x[:, 0, 5], x[:, 1, 9] = 0.0, 0.0
    x[:, first, 20:64] = -16.0                           # more mass elsewhere: the lower score
    scores = np.full((S, W), np.float32(-1000.0))
    ref, parents, tokens, _ = B.select(x.double().numpy()[:1], scores[:1], 2)
    assert ref[0, 0] > ref[0, 1] and np.float32(ref[0, 0]) == np.float32(ref[0, 1]) == -1000
    assert parents[0].tolist() == [1 - first, first]
    sc, par, tok = select(x, scores, 2)
    assert (sc == -1000).all()
    assert par.tolist() == parents.tolist() * S and tok.tolist() == tokens.tolist() * S


@pytest.mark.parametrize("kind", ["normal", "steps", "close"])
@pytest.mark.parametrize("dn", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("S,W,V,k", [(2, 4, 32000, 32), (150, 3, 700, 24), (3, 8, 20001, 64), (1, 2, 90, 60)])
def test_a_beams_candidates_come_by_their_logits(S, W, V, k, dn, kind):
    """Within a beam the log-sum-exp cancels: what is chosen of it are its largest logits, the
    lower token first where they are equal, whatever the sum's error; scores do not rise."""
    rng = np.random.default_rng(V + k)
    x = rng.standard_normal((S, W, V)).astype(np.float32)
    x = {"normal": x * 3, "steps": np.round(x), "close": 5 + x * 1e-6}[kind]
    x = torch.from_numpy(x.astype(np.float32)).to(DT[dn])
    sc, par, tok = select(x, rng.standard_normal((S, W)).astype(np.float32) - 10, k)
    assert np.isfinite(sc).all() and (np.diff(sc, axis=1) <= 0).all()
    xd = x.double().numpy()
    for s in range(S):
        for w in range(W):
            mine = tok[s, par[s] == w]
            assert np.array_equal(mine, np.lexsort((np.arange(V), -xd[s, w]))[:len(mine)])


@pytest.mark.parametrize("dn", ["f16", "f32"])
def test_the_logarithm_of_the_sum(dn):
    """Rows of n equal logits, n = 1 .. 4096, at the scores fp32(log n): what is left of
    score - log n, 2e-7 at most, shows the logarithm's own error, as the sum n is exact.
    It is to be right to 2^-29: the quotient of its series, at most 2^-5, is rounded by
    2^-30 at most, the terms left out are below 2^-32, the roundings of the rest (numbers
    below 2^-11) a few 2^-35; the result's own rounding is 2^-24 of it."""
    V = 4096
    n = np.arange(1, V + 1)
    x = torch.full((V, 1, V), -math.inf, dtype=DT[dn])
    x[torch.from_numpy(n)[:, None, None] > torch.arange(V)] = 0.75
    scores = np.log(n).astype(np.float32)[:, None]
    sc, par, tok = select(x, scores, 1)
    exact = scores[:, 0].astype(np.float64) - np.log(n.astype(np.float64))
    err = np.abs(sc[:, 0] - exact)
    assert not par.any() and not tok.any() and sc[0, 0] == 0
    assert err.max() <= 2.0 ** -29 + 2.0 ** -24 * np.abs(exact).max(), (n[err.argmax()], err.max())


def test_the_logarithm_near_one():
    """One more candidate d below the best: score - log(1 + e^-d), d = 2 .. 20.  2^x is right
    to 2^-22 of itself, its argument (d log2 e, rounded twice) to d 2^-23 of it: e^-d (2^-21 + d
    2^-22) in all; the sum is rounded by 2^-24, its logarithm is off by 2^-29."""
    d = np.linspace(2, 20, 4001).astype(np.float32)
    x = torch.full((len(d), 1, 8), -math.inf)
    x[:, 0, 2] = 1.0
    x[:, 0, 5] = 1.0 - torch.from_numpy(d)
    gap = 1.0 - x[:, 0, 5].double().numpy()
    exact = np.log1p(np.exp(-gap))
    scores = exact.astype(np.float32)[:, None]
    sc, _, tok = select(x, scores, 1)
    left = scores[:, 0].astype(np.float64) - exact
    tol = np.exp(-gap) * (2.0 ** -21 + gap * 2.0 ** -22) + 2.0 ** -24 + 2.0 ** -29 + 2.0 ** -24 * np.abs(left)
    assert (tok == 2).all() and (np.abs(sc[:, 0] - left) <= tol).all(), float((np.abs(sc[:, 0] - left) / tol).max())
