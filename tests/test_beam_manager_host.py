"""The block manager under a beam request: the recipe of the header, with the
reordering's reference in the device's place."""
import numpy as np
import pytest

from tests import _beam_manager as M
from tests import _beam_ref as B


@pytest.mark.parametrize("prefix_caching", [False, True])
@pytest.mark.parametrize("n0,W", [(1, 2), (16, 3), (21, 4), (47, 8), (32, 1)])
def test_every_row_keeps_its_history(n0, W, prefix_caching):
    max_blocks, steps = 8, 60
    pool = np.full((1 + W * max_blocks, 16), -9)

    def copy(src, dst):
        pool[dst] = pool[src]

    def write(blocks, slot, tokens):
        assert len(set(blocks)) == len(blocks)           # no two rows write into one block
        pool[blocks, slot] = tokens

    def reorder(tables, n, parents):
        new, copies = B.reorder(tables[None], [n], parents[None])
        for src, dst, t in copies:
            pool[dst, :t] = pool[src, :t]
        return new[0]

    tables, n, hist = M.search(n0, W, steps, n0 + W, prefix_caching, copy, write, reorder, max_blocks)
    for w in range(W):
        i = np.arange(n)
        assert pool[tables[w, i // 16], i % 16].tolist() == hist[w]
