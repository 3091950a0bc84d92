"""Sizes at the ends of 32 bits in the calls of cross attention and beam search
(no GPU needed: a refused call reaches no CUDA call)."""
import pytest

from tests.test_beam_cross_host import INVALID, REORDER, lib  # noqa: F401


@pytest.mark.parametrize("W", [1, 8])
def test_reorder_refuses_tables_whose_tokens_pass_32_bits(lib, W):  # noqa: F811
    """16 tokens a block: 2^27 blocks are 2^31 tokens, which a length cannot count."""
    for mb in (1 << 27, 1 << 30):
        kw = dict(REORDER, S=1, W=W, mb=mb)
        kw["out"] = kw["bt"]
        assert lib.pa_beam_reorder(*kw.values(), None) == INVALID
