"""Sizes at the ends of 32 bits in the calls of cross attention and beam search
(no GPU needed: a refused call reaches no CUDA call)."""
import pytest

import paged_kv_attention_decode_gb300 as pa
from tests._stand_in import StandIn
from tests.test_beam_cross_host import I32, INVALID, REORDER, cross_args, lib, select_args, z  # noqa: F401


@pytest.mark.parametrize("W", [1, 8])
def test_reorder_refuses_tables_whose_tokens_pass_32_bits(lib, W):  # noqa: F811
    """16 tokens a block: 2^27 blocks are 2^31 tokens, which a length cannot count."""
    for mb in (1 << 27, 1 << 30):
        kw = dict(REORDER, S=1, W=W, mb=mb)
        kw["out"] = kw["bt"]
        assert lib.pa_beam_reorder(*kw.values(), None) == INVALID


@pytest.mark.parametrize("past", [2 ** 31, 2 ** 32, 2 ** 32 + 30, 2 ** 40, 2 ** 63 - 1])
def test_bounds_of_lengths_past_32_bits_are_the_largest(monkeypatch, past):
    """Not their low bits, below which sequences would be refused on the device."""
    s = StandIn(monkeypatch)
    pa.paged_cross_attention(**cross_args(cu_q_lens=z(4, dtype=I32), max_q_len=past, max_enc_len=past))
    (_, a), = s.calls
    assert a[10:12] == (2 ** 31 - 1, 2 ** 31 - 1)
    s.calls.clear()
    pa.paged_cross_attention(**cross_args(cu_q_lens=z(4, dtype=I32), max_q_len=-past, max_enc_len=-past))
    assert s.calls[0][1][10] < 0 and s.calls[0][1][11] < 0             # (refused by the library)


@pytest.mark.parametrize("num_out", [2 ** 31, 2 ** 32 + 4, -2 ** 32 + 4])
def test_numbers_of_results_past_32_bits_are_refused(monkeypatch, num_out):
    s = StandIn(monkeypatch)
    with pytest.raises(pa.PagedAttnError, match="num_out"):
        pa.beam_select(**select_args(num_out=num_out))
    assert not s.calls
