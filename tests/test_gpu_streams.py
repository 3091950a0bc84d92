"""Calls on a stream that is not torch's current one: their scratch stays theirs
while the current stream allocates and overwrites memory of the same sizes."""
import math

import numpy as np
import pytest
import torch

import paged_kv_attention_decode_gb300 as pa

pytestmark = pytest.mark.gpu
DEV = "cuda"
HQ, HKV, D = 16, 2, 128


def case(kind, seed):
    """(call(**kw), scratch bytes) of an attention call with partials, and with a
    chunk where it is a varlen one."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    varlen = kind.startswith("prefill")
    lens, qlens = ([900, 2000, 37, 300], [1, 5, 3, 300]) if varlen else ([900, 2000, 37, 1500], [1] * 4)
    used = [(n + 15) // 16 for n in lens]
    NB = sum(used) + 2
    perm = torch.randperm(NB, generator=g, device=DEV).to(torch.int32)
    bt = torch.zeros(len(lens), max(used), dtype=torch.int32, device=DEV)
    at = 0
    for b, u in enumerate(used):
        bt[b, :u] = perm[at:at + u]
        at += u
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(qlens)]), dtype=torch.int32, device=DEV)
    q = torch.randn(sum(qlens), HQ, D, generator=g, device=DEV).to(torch.bfloat16)
    k, v = (torch.randn(NB * 16, HKV, D, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    slots = torch.arange(NB * 16, device=DEV)
    what = kind.split("_")[1] if "_" in kind else "16"
    if what == "fp8":
        pools = [torch.zeros(NB, HKV, 16, D, dtype=torch.uint8, device=DEV) for _ in range(2)]
        pa.paged_kv_write_fp8(k, v, *pools, slots, 1 / 16, 1 / 16)
    elif what == "fp4":
        pools = [torch.zeros(NB, HKV, pa.fp4_tile_bytes(D), dtype=torch.uint8, device=DEV) for _ in range(2)]
        pa.paged_kv_write_fp4(k, v, *pools, slots, 1 / 256, 1 / 256)
    else:
        pools = [x.view(NB, 16, HKV, D) for x in (k, v)]
    scales = {"fp8": (1 / 16, 1 / 16), "fp4": (1 / 256, 1 / 256)}.get(what, ())
    mods = dict(softcap=20.0, window=700) if what == "mod" else {}
    sc, mx = 1 / math.sqrt(D), max(lens)
    name = "paged_attention_" + kind
    if varlen:
        size = (len(lens), sum(qlens), HQ)
        n = {"16": lambda: pa.prefill_workspace_bytes(*size, D, mx),
             "mod": lambda: pa.prefill_mod_workspace_bytes(*size, HKV, D, mx),
             "fp8": lambda: pa.prefill_fp8_workspace_bytes(*size, HKV, D, mx, bt.shape[1], 300),
             "fp4": lambda: pa.prefill_fp4_workspace_bytes(*size, HKV, D, mx, bt.shape[1], 300)}[what]()
        extra = dict(chunk_kv_tokens=300) if scales else mods
        return lambda **kw: getattr(pa, name)(q, *pools, bt, sl, cu, sc, *scales, max(qlens), mx, **extra, **kw), n
    part = pa.decode_partition_for(len(lens), HQ, HKV, mx) if what in ("fp4", "mod") else 0
    n = pa.decode_workspace_bytes(len(lens), HQ, D, mx, part)
    return lambda **kw: getattr(pa, name)(q, *pools, bt, sl, sc, *scales, mx, **mods, **kw), n


@pytest.mark.parametrize("kind", ["decode", "prefill", "decode_fp8", "prefill_fp8", "decode_fp4", "prefill_fp4",
                                  "decode_mod", "prefill_mod"])
@pytest.mark.parametrize("as_handle", [False, True])
def test_scratch_of_a_call_on_a_given_stream(kind, as_handle):
    call, nbytes = case(kind, seed=len(kind))
    alone = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    given = side.cuda_stream if as_handle else side
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)            # the call's kernels wait behind this (about 10 ms)
        outs = [call(stream=given) for _ in range(2)]
        # meanwhile the current stream makes and fills tensors of the scratch's size
        fill = [torch.full((nbytes,), 0xFF, dtype=torch.uint8, device=DEV) for _ in range(4)]
        torch.cuda.synchronize()
        assert all(torch.equal(o, alone) for o in outs)
        del outs, fill
    assert pa.device_error() == 0


def test_results_dropped_on_the_callers_stream():
    """A result that the caller's stream still reads when it is dropped is not
    handed out again before."""
    call, _ = case("decode_mod", seed=3)
    alone = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = call(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(20_000_000)
    kept = out.clone()                               # waits behind the sleep
    size, dt = out.shape, out.dtype
    del out
    with torch.cuda.stream(side):
        fill = [torch.full(size, float("nan"), dtype=dt, device=DEV) for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(kept, alone) and len(fill) == 4


def test_appends_and_lengths_on_a_given_stream():
    """The maximum length, and the outputs, of calls that follow work of their own
    stream."""
    side = torch.cuda.Stream()
    T, rot = 40, 128
    g = torch.Generator(device=DEV).manual_seed(1)
    q, k, v = (torch.randn(T, h, D, generator=g, device=DEV).to(torch.bfloat16) for h in (HQ, HKV, HKV))
    ang = torch.arange(T, device=DEV)[:, None] * 10000.0 ** (-torch.arange(rot // 2, device=DEV) / (rot // 2))
    cs = torch.cat([ang.cos(), ang.sin()], 1).float()
    pos, bt = torch.arange(T, device=DEV), torch.arange(3, dtype=torch.int32, device=DEV)[None].contiguous()
    pools = [torch.zeros(3, 16, HKV, D, dtype=torch.bfloat16, device=DEV) for _ in range(2)]

    def steps(sl, **kw):
        cu = torch.tensor([0, T], dtype=torch.int32, device=DEV)
        torch.cuda.synchronize()
        if kw:
            with torch.cuda.stream(side):
                torch.cuda._sleep(20_000_000)
                sl += T                                  # the lengths of this step, behind the sleep
        else:
            sl += T
        slots = pa.slot_mapping(bt, sl, cu, T, 3, **kw)
        qr = pa.paged_rope_kv_write(q, k, v, *pools, slots, pos, cs, **kw)
        with torch.cuda.stream(kw.get("stream", torch.cuda.current_stream())):
            last = qr[-1:].contiguous()
        out = pa.paged_attention_decode_mod(last, *pools, bt, sl, 0.1, window=30, **kw)
        kg, _ = pa.paged_kv_gather(*pools, bt, sl, T, **kw)
        torch.cuda.synchronize()
        return slots, qr, out, kg

    a = steps(torch.zeros(1, dtype=torch.int32, device=DEV))
    b = steps(torch.zeros(1, dtype=torch.int32, device=DEV), stream=side)
    assert all(torch.equal(x, y) for x, y in zip(a, b)) and b[3].shape[0] == T
    assert pa.device_error() == 0


@pytest.mark.parametrize("kind", ["decode_fp4", "prefill_mod"])
def test_a_forked_stream_inside_a_capture(kind):
    """Two calls of a captured step, one of them on a forked stream given by
    `stream`, each with scratch of its own from the graph's pool."""
    (one, _), (two, _) = case(kind, seed=5), case(kind, seed=6)
    want = [one(), two()]
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        a, b = one(stream=side), two()
        one(stream=side)                                       # (a result dropped inside the capture)
        main.wait_stream(side)
    for _ in range(3):
        a.zero_(), b.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])
    assert pa.device_error() == 0
