"""Cross attention and beam search: what one kernel of a chain writes and the next
reads, under programmatic dependent launch, is read with plain loads behind the
wait (the lists of test_plan_loads_host.py for these chains)."""
import os
import re

import pytest

from tests.test_plan_loads_host import CSRC, SOURCES, code

# Arrays written between dependently launched kernels: the selection's pieces for
# its join; the plan, and the items dealt out, for the chunk kernel; the uniform
# rows for the plan and the chunk kernel; tables and pools that a reordering or a
# selection in place goes on from.
WRITTEN = ["sums", "all_sums", "groups", "deal", "offsets", "order", "seq_of_pair", "cu", "tables", "tables_out", "parents",
           "scores", "finished", "logits", "out_scores", "out_parents", "out_tokens", "out_finished"]
# Members that only the caller's earlier work writes, which is complete behind the wait.
INPUTS = {"out", "q", "block_tables", "seq_lens", "cu_q_lens", "err"}
MINE = ["pa_beam.cu", "pa_cross.cu"]


@pytest.mark.parametrize("name", SOURCES)
def test_no_read_only_load_of_what_the_chains_write(name):
    text = code(name)
    for args in re.findall(r"__ldg\(((?:[^()]|\([^()]*\))*)\)", text):
        assert not set(re.findall(r"\w+", args)) & set(WRITTEN), f"{name}: __ldg({args})"
    for w in WRITTEN:
        assert not re.search(r"const\s+\w+\*\s*__restrict__\s+%s\b" % w, text), f"{name}: {w}"


@pytest.mark.parametrize("name", MINE)
def test_no_read_only_load_at_all(name):
    text = code(name)
    assert not re.search(r"__restrict__|__ldg|ld\.global\.nc|ldg_stream", text)


def test_the_plan_of_chunks_reads_rows_that_a_kernel_may_have_written():
    """uniform_rows_kernel writes cu_q_lens right before it, under dependent launch."""
    text = code("pa_prefill_tc.cu")
    head = re.search(r"cross_plan_kernel\((.*?)\)\s*\{", text, re.S).group(1)
    assert "cu_q_lens" in head and "__restrict__" not in head and "__ldg" not in head
    body = text[text.index("cross_plan_kernel("):]
    assert 0 < body.index("pdl_wait();") < body.index("cu_q_lens[b]")


@pytest.mark.parametrize("struct", ["CrossParams", "BeamSelectParams", "BeamReorderParams"])
def test_the_lists_are_the_members_of_the_structs(struct):
    with open(os.path.join(CSRC, "pa_internal.h")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    body = re.search(r"struct %s \{(.*?)\n\};" % struct, text, re.S).group(1)
    members = re.findall(r"\*\s*(\w+);", body)
    assert members
    for member in members:
        assert member in INPUTS or member in WRITTEN, (struct, member)
    arrays = re.findall(r"\*\s*(\w+)\[", body)               # the pools: read and written by the copies
    assert arrays == (["k", "v"] if struct == "BeamReorderParams" else [])


@pytest.mark.parametrize("kernel", ["beam_pieces_kernel", "beam_join_kernel", "beam_few_kernel", "beam_copy_kernel",
                                    "beam_tables_kernel"])
def test_every_kernel_of_the_chains_waits(kernel):
    text = code("pa_beam.cu")
    at = re.search(r"%s\(const [^)]*\) \{" % kernel, text).end()
    body = text[at:text.index("\n}", at)]
    assert "pdl_wait();" in body
