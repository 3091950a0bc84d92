"""Attention over a 4-bit cache (decode, verify rows, prefill chunks) against a
64-bit reference over the values that the cache's bytes stand for."""
import math

import numpy as np
import pytest
import torch

import paged_kv_attention_decode_gb300 as pa
from tests import _ref64 as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
KS, VS = 1 / 256, 1 / 128


def build(lens, qlens, Hq, Hkv, D, dt, seed, qscale=1.0):
    """Pools of quantised N(0, 1) rows with scattered blocks; slots that no
    sequence covers (tails of last blocks too) hold random codes and NaN scales."""
    rng = np.random.default_rng(seed)
    used = [(int(n) + 15) // 16 for n in lens]
    NB = sum(used) + 3
    perm = rng.permutation(NB)
    tables = rng.integers(-5, NB + 5, (len(lens), max(1, max(used))))
    live = np.zeros((NB, 16), bool)
    at = 0
    for b, u in enumerate(used):
        tables[b, :u] = perm[at:at + u]
        at += u
        for j in range(int(lens[b])):
            live[tables[b, j // 16], j % 16] = True
    pools = []
    for isv, sc in ((False, KS), (True, VS)):
        codes, s = R.quantise_fp4(rng.standard_normal((NB, 16, Hkv, D)).astype(np.float32), sc)
        codes[~live] = rng.integers(0, 16, codes[~live].shape)
        s[~live] = 127
        pools.append(R.pack_tiles(codes, s, isv))
    T = int(sum(qlens))
    q = (torch.randn(T, Hq, D, generator=torch.Generator().manual_seed(seed)) * qscale).to(dt)
    return q, pools, tables.astype(np.int32)


def put(*arrays):
    return [(a if isinstance(a, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(a))).to(DEV) for a in arrays]


def check(out, q, pools, tables, lens, qlens, scale, bad=()):
    kv = [R.tile_values(p, isv, s) for p, isv, s in zip(pools, (False, True), (KS, VS))]
    ref, A, smax, cnt = R.attention(q.double().numpy(), *kv, tables, lens, qlens, scale, bad=bad)
    tol = R.bound(ref, A, smax, cnt, 6 * 448 * VS, q.dtype, torch.float16)
    got = out.double().cpu().numpy()
    assert np.all(np.isfinite(got))
    worst = np.max(np.abs(got - ref) / tol) if got.size else 0
    assert worst <= 1, worst


def decode(q, pools, tables, lens, scale, **kw):
    qd, kd, vd, td, ld = put(q, *pools, tables, np.asarray(lens, np.int32))
    out = pa.paged_attention_decode_fp4(qd, kd, vd, td, ld, scale, KS, VS, max_seq_len=int(max(lens)), **kw)
    torch.cuda.synchronize()
    return out


def step(q, pools, tables, lens, qlens, scale, **kw):
    cu = np.concatenate([[0], np.cumsum(qlens)]).astype(np.int32)
    qd, kd, vd, td, ld, cd = put(q, *pools, tables, np.asarray(lens, np.int32), cu)
    out = pa.paged_attention_prefill_fp4(qd, kd, vd, td, ld, cd, scale, KS, VS, int(max(qlens)), int(max(lens)), **kw)
    torch.cuda.synchronize()
    return out


LENS = [1, 2, 15, 16, 17, 31, 33, 100, 511, 512, 513, 1025, 700]


@pytest.mark.parametrize("Hq,Hkv,D,dn", [(4, 4, 128, "f16"), (4, 4, 128, "bf16"), (3, 3, 64, "f16"), (8, 1, 64, "bf16"),
                                         (8, 2, 128, "f16"), (16, 2, 128, "bf16"), (10, 2, 64, "bf16"),
                                         (7, 1, 128, "f16"), (24, 2, 128, "f16"), (64, 1, 128, "bf16"),
                                         (40, 2, 64, "f16")])
def test_decode(Hq, Hkv, D, dn):
    q, pools, tables = build(LENS, [1] * len(LENS), Hq, Hkv, D, DT[dn], seed=Hq + D)
    out = decode(q, pools, tables, LENS, 1 / math.sqrt(D))
    check(out, q, pools, tables, LENS, [1] * len(LENS), 1 / math.sqrt(D))
    assert pa.device_error() == 0


@pytest.mark.parametrize("part", [16, 64, 1024])
def test_decode_partitions(part):
    q, pools, tables = build(LENS, [1] * len(LENS), 8, 2, 128, torch.bfloat16, seed=part)
    out = decode(q, pools, tables, LENS, 0.09, partition_size=part)
    check(out, q, pools, tables, LENS, [1] * len(LENS), 0.09)


@pytest.mark.parametrize("qscale", [1e-30, 1e-4, 300.0])
@pytest.mark.parametrize("scale", [0.09, -0.05, 0.0])
def test_decode_query_magnitudes(qscale, scale):
    # bf16 queries far outside fp16's range enter exactly (a power of two per column)
    lens = [40, 300]
    q, pools, tables = build(lens, [1, 1], 8, 2, 128, torch.bfloat16, seed=4, qscale=qscale)
    q[0, 0] = 0
    q[1, 3, 5] *= 1000
    out = decode(q, pools, tables, lens, scale)
    check(out, q, pools, tables, lens, [1, 1], scale)


def test_moving_reference():
    # scores that pass the running reference by more than 2^8 block after block
    lens = [200]
    q, pools, tables = build(lens, [1], 4, 1, 64, torch.float16, seed=8)
    q = torch.ones_like(q)
    codes, s = R.unpack_tiles(pools[0], False)
    for j in range(200):
        codes[tables[0, j // 16], j % 16] = 2 + min(5, j // 33)      # rising keys
        s[tables[0, j // 16], j % 16] = 0x50
    pools[0] = R.pack_tiles(codes, s, False)
    for scale in (2.0, -2.0):
        out = decode(q, pools, tables, lens, scale)
        check(out, q, pools, tables, lens, [1], scale)


def test_empty_and_bad_rows():
    lens = [30, 0, 50, 64]
    q, pools, tables = build(lens, [1] * 4, 8, 4, 128, torch.float16, seed=2)
    tables[2, 1] = 10 ** 6                    # tokens 16 .. 31 contribute nothing
    qd, kd, vd, td, ld = put(q, *pools, tables, np.asarray(lens, np.int32))
    out = torch.full_like(qd, 3.0)
    pa.paged_attention_decode_fp4(qd, kd, vd, td, ld, 0.1, KS, VS, 64, out=out)
    assert pa.device_error() == 1
    check(out, q, pools, tables, lens, [1] * 4, 0.1)
    assert torch.all(out[1] == 0)
    tables[2] = -1                            # a row whose every block is bad
    td = put(tables)[0]
    pa.paged_attention_decode_fp4(qd, kd, vd, td, ld, 0.1, KS, VS, 64, out=out)
    assert pa.device_error() == 1
    assert torch.all(out[2] == 0)
    # a length above the stated maximum is rejected as in the other decodes
    pa.paged_attention_decode_fp4(qd, kd, vd, td, ld, 0.1, KS, VS, 50, out=out)
    assert pa.device_error() & 4 and torch.all(out[3] == 0)


@pytest.mark.parametrize("Hq,Hkv,D,dn", [(4, 4, 128, "bf16"), (8, 2, 128, "f16"), (16, 1, 64, "bf16"),
                                         (24, 3, 128, "bf16"), (6, 2, 64, "f16")])
def test_verify_and_decode_rows(Hq, Hkv, D, dn):
    lens, qlens = [5, 17, 600, 1024, 33, 2, 1300, 8], [5, 8, 3, 1, 2, 2, 7, 8]
    q, pools, tables = build(lens, qlens, Hq, Hkv, D, DT[dn], seed=Hq * D)
    out = step(q, pools, tables, lens, qlens, 1 / math.sqrt(D))
    check(out, q, pools, tables, lens, qlens, 1 / math.sqrt(D))
    assert pa.device_error() == 0


STEP = [(300, 300), (500, 37), (213, 9), (400, 150), (50, 2), (700, 8), (90, 4), (549, 1), (16, 1), (1, 1), (129, 128)]


@pytest.mark.parametrize("Hq,Hkv,D,dn", [(4, 4, 128, "f16"), (8, 2, 128, "bf16"), (6, 2, 64, "bf16"),
                                         (16, 1, 64, "f16")])
def test_varlen_step(Hq, Hkv, D, dn):
    lens, qlens = zip(*STEP)
    q, pools, tables = build(lens, qlens, Hq, Hkv, D, DT[dn], seed=Hq + Hkv)
    out = step(q, pools, tables, lens, qlens, 1 / math.sqrt(D))
    # (chunks: P in the query's type; the fp16 bound of `check` is for verify
    # and decode rows, so bf16 chunks get the wider one)
    kv = [R.tile_values(p, isv, s) for p, isv, s in zip(pools, (False, True), (KS, VS))]
    ref, A, smax, cnt = R.attention(q.double().numpy(), *kv, tables, lens, qlens, 1 / math.sqrt(D))
    tol = R.bound(ref, A, smax, cnt, 6 * 448 * VS, DT[dn], DT[dn])
    got = out.double().cpu().numpy()
    assert np.all(np.isfinite(got)) and np.max(np.abs(got - ref) / tol) <= 1
    assert pa.device_error() == 0
    # without a size hint the copy is sized from the arrays: the same bits
    assert torch.equal(out, step(q, pools, tables, lens, qlens, 1 / math.sqrt(D), chunk_kv_tokens=sum(lens)))


def test_chunks_that_do_not_fit_the_copy_are_skipped():
    lens, qlens = [300, 1000, 50], [300, 37, 1]
    q, pools, tables = build(lens, qlens, 8, 2, 64, torch.bfloat16, seed=6)
    cu = np.concatenate([[0], np.cumsum(qlens)]).astype(np.int32)
    qd, kd, vd, td, ld, cd = put(q, *pools, tables, np.asarray(lens, np.int32), cu)
    per = 2 * 16 * 2 * 64 * 2
    n = pa.prefill_fp4_workspace_bytes(3, int(cu[-1]), 8, 2, 64, 1000, tables.shape[1], 300)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)     # 19 + 2 blocks: the first chunk's alone
    assert n > 21 * per
    out = torch.full_like(qd, 5.0)
    pa.paged_attention_prefill_fp4(qd, kd, vd, td, ld, cd, 0.1, KS, VS, 300, 1000, out=out, workspace=ws,
                                   chunk_kv_tokens=300)
    assert pa.device_error() == 16
    assert torch.all(out[300:337] == 5.0)
    kv = [R.tile_values(p, isv, s) for p, isv, s in zip(pools, (False, True), (KS, VS))]
    ref, A, smax, cnt = R.attention(q.double().numpy(), *kv, tables, lens, qlens, 0.1)
    tol = R.bound(ref, A, smax, cnt, 6 * 448 * VS, torch.bfloat16, torch.bfloat16)
    ok = np.r_[0:300, 337:338]
    assert np.max((np.abs(out.double().cpu().numpy() - ref) / tol)[ok]) <= 1


def test_long_context_many_partitions():
    lens = [9000, 33000]
    q, pools, tables = build(lens, [1, 1], 2, 1, 64, torch.bfloat16, seed=12)
    out = decode(q, pools, tables, lens, 0.125)
    check(out, q, pools, tables, lens, [1, 1], 0.125)


def test_pool_past_4_gib():
    """Tiles past 2^32 bytes of a pool: the last blocks of a large pool."""
    Hkv, D = 8, 128
    tile = pa.fp4_tile_bytes(D)
    NB = (1 << 32) // (Hkv * tile) + 40
    lens = [100, 37]
    q, pools, tables = build(lens, [1, 1], 16, Hkv, D, torch.float16, seed=13)
    n = pools[0].shape[0]
    big = []
    for p in pools:
        x = torch.full((NB, Hkv, tile), 0x7F, dtype=torch.uint8, device=DEV)
        x[NB - n:] = torch.from_numpy(p).to(DEV)
        big.append(x)
    far = np.where((tables >= 0) & (tables < n), tables + NB - n, tables).astype(np.int32)
    qd, td, ld = put(q, far, np.asarray(lens, np.int32))
    out = pa.paged_attention_decode_fp4(qd, *big, td, ld, 0.1, KS, VS, 100)
    check(out, q, pools, tables, lens, [1, 1], 0.1)
    # the writer reaches the last slot too
    k = torch.randn(1, Hkv, D, dtype=torch.float16, device=DEV)
    pa.paged_kv_write_fp4(k, k, *big, torch.tensor([NB * 16 - 1], device=DEV), KS, VS)
    c, s = R.quantise_fp4(k.float().cpu().numpy(), KS)
    got, gs = R.unpack_tiles(big[0][-1:].cpu().numpy(), False)
    assert np.array_equal(got[0, 15], c[0]) and np.array_equal(gs[0, 15], s[0])
    assert pa.device_error() == 0


def test_steps_back_to_back_on_one_workspace():
    """Steps that differ in their chunks, queued on one workspace without a
    pause and replayed from a graph: each gives what it gives alone, bit for
    bit (the plans of a step may only start once the step before is done)."""
    Hq, Hkv, D = 8, 2, 128
    steps = []
    for i, (lens, qlens) in enumerate((([700, 40, 333], [600, 9, 1]), ([64, 900, 17, 1000], [1, 4, 17, 1]),
                                       ([1500, 1500], [1400, 1]))):
        q, pools, tables = build(lens, qlens, Hq, Hkv, D, torch.bfloat16, seed=90 + i)
        cu = np.concatenate([[0], np.cumsum(qlens)]).astype(np.int32)
        steps.append(put(q, *pools, tables, np.asarray(lens, np.int32), cu) + [max(qlens), max(lens), sum(lens)])
    need = max(pa.prefill_fp4_workspace_bytes(s[4].numel(), s[0].shape[0], Hq, Hkv, D, s[7], s[3].shape[1],
                                              s[8]) for s in steps)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)

    def go(s, out):
        pa.paged_attention_prefill_fp4(*s[:6], 0.1, KS, VS, s[6], s[7], out=out, workspace=ws,
                                       chunk_kv_tokens=s[8])

    alone = []
    for s in steps:
        o = torch.empty_like(s[0])
        go(s, o)
        torch.cuda.synchronize()
        alone.append(o)
    outs = [[torch.full_like(s[0], float("nan")) for s in steps] for _ in range(8)]
    for row in outs:
        for s, o in zip(steps, row):
            go(s, o)
    torch.cuda.synchronize()
    assert all(torch.equal(o, a) for row in outs for o, a in zip(row, alone))
    for row in outs:
        for o in row:
            o.fill_(float("nan"))
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        for row in outs:
            for s, o in zip(steps, row):
                go(s, o)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, a) for row in outs for o, a in zip(row, alone))
    assert pa.device_error() == 0


@pytest.mark.parametrize("verify", [False, True])
def test_decode_and_verify_calls_back_to_back_on_one_workspace(verify):
    """Calls without chunks, whose plan starts while the call before still runs:
    other lengths, batch sizes and partitions each time, one workspace, queued
    without a pause and replayed from a graph.  Each gives what it gives alone."""
    Hq, Hkv, D = 8, 2, 128
    rng = np.random.default_rng(17)
    calls = []
    for i, (B, hi, part) in enumerate(((40, 900, 64), (3, 3000, 16), (70, 60, 0), (1, 2500, 128), (25, 1500, 64))):
        lens = [int(n) for n in rng.integers(8, hi, B)]
        qlens = [int(c) for c in rng.integers(1, 9, B)] if verify else [1] * B
        q, pools, tables = build(lens, qlens, Hq, Hkv, D, torch.bfloat16, seed=200 + i)
        cu = np.concatenate([[0], np.cumsum(qlens)]).astype(np.int32)
        d = put(q, *pools, tables, np.asarray(lens, np.int32), cu)
        mx = max(lens)
        need = pa.prefill_mod_workspace_bytes(B, int(cu[-1]), Hq, Hkv, D, mx) if verify else \
            pa.decode_workspace_bytes(B, Hq, D, mx, part or pa.decode_partition_for(B, Hq, Hkv, mx))
        calls.append((d, mx, part, need))
    ws = torch.empty(max(c[3] for c in calls), dtype=torch.uint8, device=DEV)

    def go(c, out):
        d, mx, part, _ = c
        if verify:
            pa.paged_attention_prefill_fp4(*d, 0.1, KS, VS, 8, mx, out=out, workspace=ws)
        else:
            pa.paged_attention_decode_fp4(*d[:5], 0.1, KS, VS, mx, out=out, partition_size=part, workspace=ws)

    alone = []
    for c in calls:
        o = torch.empty_like(c[0][0])
        go(c, o)
        torch.cuda.synchronize()
        alone.append(o)
    outs = [[torch.full_like(c[0][0], float("nan")) for c in calls] for _ in range(12)]
    for row in outs:
        for c, o in zip(calls, row):
            go(c, o)
    torch.cuda.synchronize()
    assert all(torch.equal(o, a) for row in outs for o, a in zip(row, alone))
    for row in outs:
        for o in row:
            o.fill_(float("nan"))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for row in outs:
            for c, o in zip(calls, row):
                go(c, o)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, a) for row in outs for o, a in zip(row, alone))
    assert pa.device_error() == 0
