"""What a plan kernel writes is read with plain loads: a kernel launched with
programmatic dependent launch may be resident while the plan still writes, and
the read-only path (`__ldg`, or a `const __restrict__` pointer) asks for data
that no one writes during the kernel's whole life."""
import os
import re

import pytest

from paged_kv_attention_decode_gb300 import _binding

CSRC = os.path.join(os.path.dirname(_binding.__file__), "csrc")
# the arrays that plans (and the kernels between a plan and its reader) write
WRITTEN = ["units", "unit_count", "work_counter", "row_base", "rows", "row_count", "split", "decode_units", "ws_m",
           "ws_l", "ws_acc", "plan", "order", "seq_of_pair", "offsets", "hdr", "chunk_seq", "chunk_base", "table",
           "k16", "v16"]
SOURCES = sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh")))


def code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", SOURCES)
def test_no_read_only_load_of_what_a_plan_writes(name):
    text = code(name)
    for args in re.findall(r"__ldg\(((?:[^()]|\([^()]*\))*)\)", text):
        names = set(re.findall(r"\w+", args))
        assert not names & set(WRITTEN), f"{name}: __ldg({args})"
    for w in WRITTEN:
        assert not re.search(r"const\s+\w+\*\s*__restrict__\s+%s\b" % w, text), f"{name}: {w}"


def test_the_lists_are_the_members():
    """Every pointer of the parameter structs is known here as written or as an input."""
    with open(os.path.join(CSRC, "pa_internal.h")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    inputs = {"out", "q", "block_tables", "seq_lens", "cu_q_lens", "err", "k_pool", "v_pool", "slopes", "q_out", "key",
              "value", "k_cache", "v_cache", "positions", "cos_sin", "slots", "k_codes", "v_codes", "src_tables"}
    for struct in ("ScoreMod", "DecodeParams", "PrefillParams", "AppendParams", "Fp8Copy"):
        body = re.search(r"struct %s \{(.*?)\n\};" % struct, text, re.S).group(1)
        for member in re.findall(r"\*\s*(\w+);", body):
            assert member in inputs or member in WRITTEN, (struct, member)
