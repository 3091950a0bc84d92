"""Rotate-and-append and the attention that follows, as a serving loop runs
them: a prompt in chunks, then decode and verify steps, over 16-bit, FP8 and
4-bit caches; captured in a graph and replayed; on side streams at once.  The
reference keeps its own copy of the cache in 64 bits."""
import math

import numpy as np
import pytest
import torch

import paged_kv_attention_decode_gb300 as pa
from tests import _ref64 as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
SCALE4, SCALE8 = 1 / 256, 1 / 16


def table(rot, n):
    half = rot // 2
    ang = np.arange(n)[:, None] * 10000.0 ** (-np.arange(half) / half)
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


class Loop:
    """Sequences growing step by step over one pool."""

    def __init__(self, cache, Hq, Hkv, D, dt, seed, nseq=3, max_len=400, mods=None, inter=False):
        self.cache, self.Hq, self.Hkv, self.D, self.dt, self.mods = cache, Hq, Hkv, D, dt, mods or {}
        self.inter, self.g = inter, torch.Generator().manual_seed(seed)
        self.mb = (max_len + 15) // 16
        self.NB = nseq * self.mb + 2
        self.tables = np.random.default_rng(seed).permutation(self.NB)[:nseq * self.mb].reshape(nseq, -1).astype(np.int32)
        self.lens = np.zeros(nseq, np.int32)
        shape = {"same": (self.NB, 16, Hkv, D), "fp8": (self.NB, Hkv, 16, D), "fp4": (self.NB, Hkv, 9 * D)}[cache]
        t = dt if cache == "same" else torch.uint8
        # what was never written reads as NaN
        fill = float("nan") if cache == "same" else 0x7F
        self.pools = [torch.full(shape, fill, dtype=t, device=DEV) for _ in range(2)]
        self.cs = table(D, max_len)
        self.cs_d = torch.from_numpy(self.cs).to(DEV)
        self.bt = torch.from_numpy(self.tables).to(DEV)
        self.ref = [np.zeros((self.NB, 16, Hkv, D)) for _ in range(2)]

    def inputs(self, new):
        T = int(sum(new))
        fused = torch.randn(T, (self.Hq + 2 * self.Hkv) * self.D, generator=self.g).to(self.dt)
        self.lens = self.lens + np.asarray(new, np.int32)
        pos = np.concatenate([np.arange(n - c, n) for n, c in zip(self.lens, new)]).astype(np.int64)
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        return fused, pos, cu

    def enqueue(self, fused_d, pos_d, cu_d, lens_d, new, max_len, q_out=None, out=None, workspace=None, slots=None):
        Hq, Hkv, D, T = self.Hq, self.Hkv, self.D, fused_d.shape[0]
        q = fused_d[:, :Hq * D].unflatten(1, (Hq, D))
        k = fused_d[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
        v = fused_d[:, (Hq + Hkv) * D:].unflatten(1, (Hkv, D))
        slots = pa.slot_mapping(self.bt, lens_d, cu_d, T, self.NB, out=slots)
        a = (q, k, v, *self.pools, slots, pos_d, self.cs_d)
        kw = dict(interleaved=self.inter, q_out=q_out)
        mq, sc = int(max(new)), 1 / math.sqrt(D)
        if self.cache == "same":
            q = pa.paged_rope_kv_write(*a, **kw)
            if mq == 1:
                return pa.paged_attention_decode_mod(q, *self.pools, self.bt, lens_d, sc, max_len, out=out,
                                                     workspace=workspace, **self.mods)
            return pa.paged_attention_prefill_mod(q, *self.pools, self.bt, lens_d, cu_d, sc, mq, max_len, out=out,
                                                  workspace=workspace, **self.mods)
        if self.cache == "fp8":
            q = pa.paged_rope_kv_write_fp8(*a, SCALE8, SCALE8, **kw)
            return pa.paged_attention_prefill_fp8(q, *self.pools, self.bt, lens_d, cu_d, sc, SCALE8, SCALE8, mq, max_len,
                                                  out=out, workspace=workspace, chunk_kv_tokens=3 * max_len)
        q = pa.paged_rope_kv_write_fp4(*a, SCALE4, SCALE4, **kw)
        if mq == 1:
            return pa.paged_attention_decode_fp4(q, *self.pools, self.bt, lens_d, sc, SCALE4, SCALE4, max_len, out=out,
                                                 workspace=workspace)
        return pa.paged_attention_prefill_fp4(q, *self.pools, self.bt, lens_d, cu_d, sc, SCALE4, SCALE4, mq, max_len,
                                              out=out, workspace=workspace, chunk_kv_tokens=3 * max_len)

    def reference(self, fused, pos, cu, new):
        Hq, Hkv, D = self.Hq, self.Hkv, self.D
        x = fused.float().numpy().reshape(-1, Hq + 2 * Hkv, D)
        q = torch.from_numpy(R.rope32(x[:, :Hq], self.cs, pos, D, self.inter)).to(self.dt).double().numpy()
        k = R.rope32(x[:, Hq:Hq + Hkv], self.cs, pos, D, self.inter)
        v = x[:, Hq + Hkv:]
        seq = np.repeat(np.arange(len(new)), new)
        blk, off = self.tables[seq, pos // 16], pos % 16
        for pool, rows in zip(self.ref, (k, v)):
            if self.cache == "same":
                val = torch.from_numpy(rows).to(self.dt).double().numpy()
            elif self.cache == "fp8":
                y = (rows * np.float32(1 / SCALE8)).astype(np.float32)
                val = np.copysign(R.E4M3[R.nearest_even(np.abs(y).astype(np.float64), R.E4M3[:127])], y) * SCALE8
            else:
                c, s = R.quantise_fp4(rows, SCALE4)
                val = R.E2M1[c] * np.repeat(R.E4M3[s], 16, -1) * SCALE4
            pool[blk, off] = val
        m = {k: v for k, v in self.mods.items() if k in ("softcap", "window")}
        ref, A, smax, cnt = R.attention(q, *self.ref, self.tables, self.lens, new, 1 / math.sqrt(D), **m)
        return ref, R.bound(ref, A, smax, cnt, float(np.abs(self.ref[1]).max()), self.dt, self.dt,
                            m.get("softcap", 0.0))

    def step(self, new):
        fused, pos, cu = self.inputs(new)
        d = [torch.from_numpy(a).to(DEV) if isinstance(a, np.ndarray) else a.to(DEV) for a in (fused, pos, cu, self.lens)]
        out = self.enqueue(*d, new, int(self.lens.max()))
        torch.cuda.synchronize()
        ref, tol = self.reference(fused, pos, cu, new)
        got = out.double().cpu().numpy()
        assert np.all(np.isfinite(got))
        assert np.max(np.abs(got - ref) / tol) <= 1
        assert pa.device_error() == 0


CONFIGS = [("same", 8, 2, 128, torch.bfloat16, dict(window=60, softcap=20.0), False),
           ("same", 4, 4, 64, torch.float16, dict(), True),
           ("fp8", 8, 2, 128, torch.float16, {}, False),
           ("fp4", 8, 2, 128, torch.bfloat16, {}, True), ("fp4", 3, 3, 64, torch.float16, {}, False)]


@pytest.mark.parametrize("cache,Hq,Hkv,D,dt,mods,inter", CONFIGS)
def test_prompt_then_decode_and_verify_steps(cache, Hq, Hkv, D, dt, mods, inter):
    lp = Loop(cache, Hq, Hkv, D, dt, seed=Hq * D, mods=mods, inter=inter)
    for new in ([130, 17, 40], [150, 1, 33], [1, 1, 1], [4, 1, 3], [1, 1, 1], [9, 8, 1], [1, 1, 1]):
        lp.step(new)


@pytest.mark.parametrize("cache,Hq,Hkv,D,dt,mods,inter", CONFIGS)
def test_captured_decode_step_replays(cache, Hq, Hkv, D, dt, mods, inter):
    """One graph of slot mapping, append and attention, replayed as the
    sequences grow; the eager result of the same step has the same bits."""
    lp = Loop(cache, Hq, Hkv, D, dt, seed=1 + D, mods=mods, inter=inter)
    lp.step([50, 1, 200])
    new = [1, 1, 1]
    fused, pos, cu = lp.inputs(new)
    bufs = [torch.from_numpy(a).to(DEV) if isinstance(a, np.ndarray) else a.to(DEV) for a in (fused, pos, cu, lp.lens)]
    fixed = dict(q_out=torch.empty(3, Hq, D, dtype=dt, device=DEV), out=torch.empty(3, Hq, D, dtype=dt, device=DEV),
                 workspace=torch.empty(1 << 23, dtype=torch.uint8, device=DEV),
                 slots=torch.empty(3, dtype=torch.int64, device=DEV))
    lp.enqueue(*bufs, new, 400, **fixed)
    lp.reference(fused, pos, cu, new)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lp.enqueue(*bufs, new, 400, **fixed)
    for _ in range(3):
        fused, pos, cu = lp.inputs(new)
        for b, a in zip(bufs, (fused, pos, cu, lp.lens)):
            b.copy_(torch.from_numpy(a) if isinstance(a, np.ndarray) else a)
        graph.replay()
        torch.cuda.synchronize()
        first = fixed["out"].clone()
        ref, tol = lp.reference(fused, pos, cu, new)
        assert np.max(np.abs(first.double().cpu().numpy() - ref) / tol) <= 1
        graph.replay()                                        # the same step again: the same bits
        torch.cuda.synchronize()
        assert torch.equal(first, fixed["out"])
        assert torch.equal(first, lp.enqueue(*bufs, new, 400))
    assert pa.device_error() == 0


def test_two_streams_at_once():
    """Two loops on streams of their own, each with its own workspace, give the
    bits that each gives alone."""
    def make(seed):
        lp = Loop("fp4", 8, 2, 128, torch.bfloat16, seed=seed, max_len=900)
        steps = []
        for new in ([700, 33, 90], [1, 1, 1], [3, 8, 1], [40, 1, 1], [1, 1, 1]):
            fused, pos, cu = lp.inputs(new)
            steps.append((new, [torch.from_numpy(a).to(DEV) if isinstance(a, np.ndarray) else a.to(DEV)
                                for a in (fused, pos, cu, lp.lens)]))
        return lp, steps

    alone = []
    for seed in (1, 2):
        lp, steps = make(seed)
        alone.append([lp.enqueue(*b, new, 900) for new, b in steps])
    torch.cuda.synchronize()
    loops = [make(seed) for seed in (1, 2)]
    streams = [torch.cuda.Stream() for _ in loops]
    torch.cuda.synchronize()
    both = [[], []]
    for i in range(5):
        for j, (lp, steps) in enumerate(loops):
            with torch.cuda.stream(streams[j]):
                both[j].append(lp.enqueue(*steps[i][1], steps[i][0], 900))
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert pa.device_error() == 0


def test_rows_behind_the_last_sequence_stay():
    """Query rows past cu_q_lens' end, and decode rows of length 0, as in the
    calls for the other caches."""
    for cache in ("same", "fp4"):
        lp = Loop(cache, 8, 2, 128, torch.float16, seed=5)
        fused, pos, cu = lp.inputs([20, 3, 30])
        d = [torch.from_numpy(a).to(DEV) if isinstance(a, np.ndarray) else a.to(DEV) for a in (fused, pos, cu, lp.lens)]
        pad = torch.full((53 + 6, 8, 128), 9.0, dtype=torch.float16, device=DEV)
        q = pa.paged_rope_kv_write(d[0][:, :1024].unflatten(1, (8, 128)), d[0][:, 1024:1280].unflatten(1, (2, 128)),
                                   d[0][:, 1280:].unflatten(1, (2, 128)), *lp.pools,
                                   pa.slot_mapping(lp.bt, d[3], d[2], 53, lp.NB), d[1], lp.cs_d) \
            if cache == "same" else \
            pa.paged_rope_kv_write_fp4(d[0][:, :1024].unflatten(1, (8, 128)), d[0][:, 1024:1280].unflatten(1, (2, 128)),
                                       d[0][:, 1280:].unflatten(1, (2, 128)), *lp.pools,
                                       pa.slot_mapping(lp.bt, d[3], d[2], 53, lp.NB), d[1], lp.cs_d, SCALE4, SCALE4)
        big = torch.cat([q, torch.ones(6, 8, 128, dtype=torch.float16, device=DEV)])
        if cache == "same":
            pa.paged_attention_prefill_mod(big, *lp.pools, lp.bt, d[3], d[2], 0.1, 30, 30, out=pad, window=9)
        else:
            pa.paged_attention_prefill_fp4(big, *lp.pools, lp.bt, d[3], d[2], 0.1, SCALE4, SCALE4, 30, 30, out=pad)
        torch.cuda.synchronize()
        assert torch.all(pad[53:] == 9.0) and torch.all(torch.isfinite(pad[:53]))
        assert pa.device_error() == 0
        # a padding row of a decode batch
        lens = torch.tensor([20, 0, 30], dtype=torch.int32, device=DEV)
        out = torch.full((3, 8, 128), 4.0, dtype=torch.float16, device=DEV)
        if cache == "same":
            pa.paged_attention_decode_mod(q[:3].contiguous(), *lp.pools, lp.bt, lens, 0.1, 30, out=out, window=5)
        else:
            pa.paged_attention_decode_fp4(q[:3].contiguous(), *lp.pools, lp.bt, lens, 0.1, SCALE4, SCALE4, 30, out=out)
        torch.cuda.synchronize()
        assert torch.all(out[1] == 0) and torch.all(torch.isfinite(out)) and pa.device_error() == 0
