"""cu_q_lens that falls somewhere, so that chunks would share query rows: the
sequences that begin before an earlier one's end are dropped and flagged, the
others keep their bits, and nothing is written past the workspace (the plans'
lists and the partials have room for rows that do not overlap)."""
import math

import numpy as np
import pytest
import torch

import paged_kv_attention_decode_gb300 as pa

pytestmark = pytest.mark.gpu
DEV = "cuda"
HQ, HKV, D, GUARD = 8, 2, 128, 1 << 16


def call(kind, cu, T, lens, max_q, seed=0):
    """(output with rows of 3.0 where nothing was written, error word)."""
    B, mx = len(lens), max(lens)
    g = torch.Generator(device=DEV).manual_seed(seed)
    mb = (mx + 15) // 16
    NB = 2 * mb + 5
    bt = torch.randint(0, NB, (B, mb), generator=g, device=DEV, dtype=torch.int32)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    cu_d = torch.tensor(cu, dtype=torch.int32, device=DEV)
    q = torch.randn(T, HQ, D, generator=g, device=DEV).to(torch.bfloat16)
    k, v = (torch.randn(NB * 16, HKV, D, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    slots = torch.arange(NB * 16, device=DEV)
    scales, extra, hint = (), {}, sum(n for n, a, b in zip(lens, cu, cu[1:]) if b - a > 8)
    if kind == "fp8":
        pools, scales = [torch.zeros(NB, HKV, 16, D, dtype=torch.uint8, device=DEV) for _ in range(2)], (1 / 16, 1 / 16)
        pa.paged_kv_write_fp8(k, v, *pools, slots, *scales)
    elif kind == "fp4":
        pools = [torch.zeros(NB, HKV, 9 * D, dtype=torch.uint8, device=DEV) for _ in range(2)]
        scales = (1 / 256, 1 / 256)
        pa.paged_kv_write_fp4(k, v, *pools, slots, *scales)
    else:
        pools = [x.view(NB, 16, HKV, D) for x in (k, v)]
    size = (B, T, HQ)
    if scales and max_q > 8:
        extra = dict(chunk_kv_tokens=hint)
        need = getattr(pa, f"prefill_{kind}_workspace_bytes")(*size, HKV, D, mx, mb, hint)
    elif kind in ("fp4", "mod"):
        need = pa.prefill_mod_workspace_bytes(*size, HKV, D, mx)
    else:
        need = pa.prefill_workspace_bytes(*size, D, mx)
    if kind == "mod":
        extra = dict(softcap=20.0)
    room = torch.full((need + GUARD,), 0xAB, dtype=torch.uint8, device=DEV)
    out = torch.full((T + 64, HQ, D), 3.0, dtype=torch.bfloat16, device=DEV)
    pa.device_error()
    f = getattr(pa, "paged_attention_prefill" + ("" if kind == "16" else "_" + kind))
    f(q, *pools, bt, sl, cu_d, 1 / math.sqrt(D), *scales, max_q, mx, out=out[:T], workspace=room[:need], **extra)
    torch.cuda.synchronize()
    assert torch.all(room[need:] == 0xAB) and torch.all(out[T:] == 3.0)
    return out[:T], pa.device_error()


CASES = {
    # name: (cu_q_lens, one in order with the kept sequences' rows, T, lens, max_q)
    "verify_rows": ([0, 8] * 21, [0] + [8] * 41, 8, [1500] * 41, 8),
    "chunks": ([0, 200] * 21, [0] + [200] * 41, 200, [300] * 41, 200),
    "some": ([0, 8, 20, 10, 30], [0, 8, 20, 20, 20], 30, [700, 100, 100, 90], 20),
    # sequence 1399 falls back to row 5, where 1400 begins
    "past_the_first_1024": (list(range(1400)) + [5] + list(range(1401, 1501)), list(range(1501)), 1500, [40] * 1500, 8),
}


@pytest.mark.parametrize("kind", ["16", "fp8", "fp4", "mod"])
@pytest.mark.parametrize("name", CASES)
def test_overlapping_rows_are_dropped_and_flagged(kind, name):
    cu, cu_ok, T, lens, max_q = CASES[name]
    out, err = call(kind, cu, T, lens, max_q)
    ref, ref_err = call(kind, cu_ok, T, lens, max_q)
    keep = np.r_[0:1399, 1401:1500] if name == "past_the_first_1024" else np.arange(cu_ok[-1])
    assert ref_err == 0
    assert err == 4                                        # PA_DEVERR_SEQ_LEN
    assert torch.equal(out[keep], ref[keep]) and torch.all(torch.isfinite(out[keep]))
    lost = np.setdiff1d(np.arange(T), keep)
    assert torch.all(out[lost] == 3.0)


def test_slots_of_rows_outside_and_behind():
    """Slots of a batch padded to more rows than its sequences have (-1 behind
    them), and of sequences past the rows (flagged, nothing written)."""
    bt = torch.arange(12, dtype=torch.int32, device=DEV).view(3, 4)
    sl = torch.tensor([40, 20, 64], dtype=torch.int32, device=DEV)

    def slots(cu, T):
        buf = torch.full((T + 300,), 77, dtype=torch.int64, device=DEV)
        pa.device_error()
        pa.slot_mapping(bt, sl, torch.tensor(cu, dtype=torch.int32, device=DEV), T, 12, out=buf[:T])
        torch.cuda.synchronize()
        assert torch.all(buf[T:] == 77)
        return buf[:T].tolist(), pa.device_error()

    want = [*range(38, 40), 64 + 19, *range(2 * 64 + 60, 2 * 64 + 64)]
    assert slots([0, 2, 3, 7], 7) == (want, 0)
    assert slots([0, 2, 3, 7], 500) == (want + [-1] * 493, 0)
    assert slots([0, 2, 3, 7], 5) == (want[:3] + [77] * 2, 4)       # the last sequence's rows end past the buffer
    assert slots([0, 0, 0, 0], 300) == ([-1] * 300, 0)
    made = pa.slot_mapping(bt, sl, torch.tensor([0, 2, 3, 7], dtype=torch.int32, device=DEV), 90, 12)
    assert made.tolist() == want + [-1] * 83
    assert pa.slot_mapping(bt[:0], sl[:0], torch.zeros(1, dtype=torch.int32, device=DEV), 9, 12).tolist() == [-1] * 9


def test_a_padded_step_appends_nothing_behind_its_sequences():
    """Slot mapping, rotate-and-append and attention of a step padded to a fixed
    number of rows: the caches hold the sequences' tokens and nothing else."""
    T, pad = 7, 64
    g = torch.Generator(device=DEV).manual_seed(2)
    bt = torch.arange(12, dtype=torch.int32, device=DEV).view(3, 4)
    sl, cu = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([2, 1, 4], [0, 2, 3, 7]))
    q, k, v = (torch.randn(pad, h, D, generator=g, device=DEV).to(torch.bfloat16) for h in (HQ, HKV, HKV))
    pos = torch.zeros(pad, dtype=torch.int64, device=DEV)
    cs = torch.cat([torch.ones(4, D // 2), torch.zeros(4, D // 2)], 1).to(DEV)
    junk = torch.arange(pad, device=DEV)                  # (the next tensor of this size may be this memory)
    del junk
    pools = [torch.zeros(12, 16, HKV, D, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    slots = pa.slot_mapping(bt, sl, cu, pad, 12)
    pa.paged_rope_kv_write(q, k, v, *pools, slots, pos, cs)
    torch.cuda.synchronize()
    flat = pools[1].view(-1, HKV, D)
    held = torch.tensor([0, 1, 64, *range(128, 132)], device=DEV)
    assert torch.equal(flat[held], v[:T])
    flat[held] = 0
    assert torch.all(flat == 0) and pa.device_error() == 0
