"""The bound of the many-partition cases rejects a zero output, an output that lost
or doubled a partition, and passes the exact result rounded to the output's type."""
import numpy as np
import pytest
import torch

from tests._fp4_merge import CASES, Case, drops


@pytest.mark.parametrize("name", CASES)
def test_the_bound_rejects_what_it_must(name):
    c = Case(**CASES[name])
    for b in range(2):
        ref, tol = c.result(b), c.bound(b)
        rounded = torch.from_numpy(ref).to(c.dt).double().numpy()
        assert np.all(np.abs(rounded - ref) <= tol)
        assert np.max(np.abs(ref) / tol) > 3                       # a zero row
        p, v, _, _ = c.row(b)
        at = np.arange(c.lens[b]) // c.part
        sets = drops(c, b)
        assert len(sets) > 8
        for lost in sets[::max(1, len(sets) // 15)]:
            hit = np.isin(at, list(lost))
            share = p[..., hit].sum(-1).reshape(-1, 1)             # [Hq, 1]
            part = np.einsum("hgn,nhd->hgd", p[..., hit], v[hit]).reshape(ref.shape)
            without = (ref - part) / (1 - share)
            twice = (ref + part) / (1 + share)
            for wrong in (without, twice):
                assert np.all(np.max(np.abs(wrong - ref) / tol, -1) > 1), (b, lost)   # for every head
        assert np.allclose(without, c.result(b, lost))
