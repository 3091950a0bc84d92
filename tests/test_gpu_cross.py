"""Cross attention to cached encoder states against a 64-bit reference: rows of
beams, ragged rows, long chunks, sequences without states."""
import math

import numpy as np
import pytest
import torch

import paged_kv_attention_decode_gb300 as pa
from tests import _beam_ref as B
from tests import _ref64 as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
SEQ_LEN, BLOCK_ID = 4, 1


def build(lens, qlens, Hq, Hkv, D, dt, seed, qscale=2.0):
    """Scattered blocks; every slot behind a sequence's states is NaN, the table
    entries behind its blocks are garbage."""
    rng = np.random.default_rng(seed)
    used = [(int(n) + 15) // 16 for n in lens]
    NB = sum(used) + 3
    perm = rng.permutation(NB)
    tables = rng.integers(-9, NB + 9, (len(lens), max(1, max(used))))
    live = np.zeros((NB, 16), bool)
    at = 0
    for b, u in enumerate(used):
        tables[b, :u] = perm[at:at + u]
        for j in range(int(lens[b])):
            live[perm[at + j // 16], j % 16] = True
        at += u
    pools = []
    for _ in range(2):
        x = torch.from_numpy(rng.standard_normal((NB, 16, Hkv, D)).astype(np.float32)).to(dt)
        x[torch.from_numpy(~live)] = float("nan")
        pools.append(x)
    q = torch.from_numpy((rng.standard_normal((int(sum(qlens)), Hq, D)) * qscale).astype(np.float32)).to(dt)
    return q, pools, tables.astype(np.int32)


def dev(tables, lens, qlens):
    cu = np.concatenate([[0], np.cumsum(qlens)])
    return (torch.from_numpy(tables).to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV),
            torch.tensor(cu, dtype=torch.int32, device=DEV))


def run(q, pools, tables, lens, qlens, scale, uniform=False, **kw):
    t, n, cu = dev(tables, lens, qlens)
    args = dict(max_enc_len=int(max(lens)), **kw)
    if not uniform:
        args.update(cu_q_lens=cu, max_q_len=int(max(qlens)))
    out = pa.paged_cross_attention(q.to(DEV), pools[0].to(DEV), pools[1].to(DEV), t, n, scale, **args)
    torch.cuda.synchronize()
    return out


def check(out, q, pools, tables, lens, qlens, scale):
    kv = [np.nan_to_num(p.double().numpy()) for p in pools]
    ref, A, smax, cnt = B.cross_attention(q.double().numpy(), *kv, tables, lens, qlens, scale)
    tol = R.bound(ref, A, smax, cnt, max(float(np.abs(kv[1]).max()), 1.0), q.dtype, q.dtype)
    got = out.double().cpu().numpy()
    assert np.all(np.isfinite(got))
    worst = np.max(np.abs(got - ref) / tol) if got.size else 0
    assert worst <= 1, worst
    r = 0
    for n, c in zip(lens, qlens):
        if n == 0:
            assert not got[r:r + c].any()
        r += c


LENS = [1, 0, 15, 16, 17, 100, 511, 513, 1025, 64]
HEADS = [(4, 4, 128, "f16"), (3, 3, 64, "bf16"), (8, 2, 128, "bf16"), (12, 12, 64, "f16"), (40, 2, 128, "f16"),
         (64, 1, 64, "bf16")]


@pytest.mark.parametrize("rows", [1, 2, 5, 8])
@pytest.mark.parametrize("Hq,Hkv,D,dn", HEADS)
def test_beams_of_every_request(Hq, Hkv, D, dn, rows):
    qlens = [rows] * len(LENS)
    q, pools, tables = build(LENS, qlens, Hq, Hkv, D, DT[dn], seed=Hq + rows)
    out = run(q, pools, tables, LENS, qlens, 1 / math.sqrt(D), uniform=True)
    check(out, q, pools, tables, LENS, qlens, 1 / math.sqrt(D))
    assert pa.device_error() == 0


@pytest.mark.parametrize("n", [1, 16, 31, 250, 1200, 4096, 9001])
@pytest.mark.parametrize("Hq,Hkv,rows", [(1, 1, 1), (2, 2, 4), (16, 2, 3)])
def test_one_request(Hq, Hkv, rows, n):
    """Few items: the states are split over a cluster of CTAs."""
    for D, dn in ((64, "bf16"), (128, "f16")):
        q, pools, tables = build([n], [rows], Hq, Hkv, D, DT[dn], seed=n + rows)
        out = run(q, pools, tables, [n], [rows], 1 / math.sqrt(D), uniform=True)
        check(out, q, pools, tables, [n], [rows], 1 / math.sqrt(D))
    assert pa.device_error() == 0


@pytest.mark.parametrize("Hq,Hkv,D,dn", HEADS)
def test_ragged_rows_and_chunks(Hq, Hkv, D, dn):
    """Short rows and chunks (longer than their states, too) in one call; a
    sequence may have no row."""
    lens = [300, 0, 17, 1, 129, 40, 0, 128, 700, 16]
    qlens = [9, 12, 8, 150, 0, 1, 3, 64, 33, 5]
    q, pools, tables = build(lens, qlens, Hq, Hkv, D, DT[dn], seed=Hq)
    out = run(q, pools, tables, lens, qlens, 1 / math.sqrt(D))
    check(out, q, pools, tables, lens, qlens, 1 / math.sqrt(D))
    assert pa.device_error() == 0


@pytest.mark.parametrize("rows", [9, 130])
def test_uniform_chunks(rows):
    lens = [200, 0, 1, 640]
    qlens = [rows] * 4
    q, pools, tables = build(lens, qlens, 8, 2, 64, torch.float16, seed=rows)
    out = run(q, pools, tables, lens, qlens, 0.125, uniform=True)
    check(out, q, pools, tables, lens, qlens, 0.125)
    assert pa.device_error() == 0


@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0])
def test_scales(scale):
    """Equal weights, negative scales, and scores far apart."""
    lens, qlens = [50, 333], [4, 20]
    q, pools, tables = build(lens, qlens, 4, 2, 128, torch.bfloat16, seed=3)
    out = run(q, pools, tables, lens, qlens, scale)
    check(out, q, pools, tables, lens, qlens, scale)


def test_large_scores_in_the_last_block():
    """The running maximum rises by far more than the lazy rescale allows, late."""
    lens, qlens = [1000, 1000], [3, 40]
    q, pools, tables = build(lens, qlens, 2, 2, 64, torch.float16, seed=8)
    for b in range(2):
        pools[0][tables[b, 62], 5] *= 30
    out = run(q, pools, tables, lens, qlens, 0.125)
    check(out, q, pools, tables, lens, qlens, 0.125)


def test_blocks_outside_the_pool_contribute_nothing():
    lens, qlens = [200, 90, 16, 400], [4, 20, 2, 1]
    q, pools, tables = build(lens, qlens, 4, 2, 64, torch.float16, seed=5)
    NB = pools[0].shape[0]
    tables[0, 3], tables[0, 12], tables[1, 0], tables[2, 0], tables[3, 7] = -1, NB, NB + 7, -5, 2 ** 31 - 1
    out = run(q, pools, tables, lens, qlens, 0.125)
    check(out, q, pools, tables, lens, qlens, 0.125)
    assert pa.device_error() == BLOCK_ID


def test_bad_lengths_give_zero_rows_and_a_flag():
    lens, qlens = [100, 30, 50, 20], [2, 12, 3, 9]
    q, pools, tables = build(lens, qlens, 4, 2, 64, torch.float16, seed=6)
    t, n, cu = dev(tables, lens, qlens)
    n[0], n[1] = -3, 1 << 20
    out = pa.paged_cross_attention(q.to(DEV), pools[0].to(DEV), pools[1].to(DEV), t, n, 0.125, max_enc_len=100,
                                   cu_q_lens=cu, max_q_len=12)
    torch.cuda.synchronize()
    assert pa.device_error() == SEQ_LEN
    assert not out[:14].any()
    check(out, q, pools, tables, [0, 0, 50, 20], qlens, 0.125)


def test_rows_of_no_sequence_stay():
    lens, qlens = [70, 33], [3, 11]
    q, pools, tables = build([70, 33, 0], [3, 11, 6], 4, 4, 64, torch.bfloat16, seed=9)
    t, n, cu = dev(tables[:2], lens, qlens)
    out = torch.full((20, 4, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    got = pa.paged_cross_attention(q.to(DEV), pools[0].to(DEV), pools[1].to(DEV), t, n, 0.125, max_enc_len=70,
                                   cu_q_lens=cu, max_q_len=11, out=out)
    assert got is out
    check(out[:14], q[:14], pools, tables, lens, qlens, 0.125)
    assert bool((out[14:] == 7).all())
    assert pa.device_error() == 0


@pytest.mark.parametrize("max_q", [2, 8])
def test_more_rows_than_max_q_len(max_q):
    """Not written, and flagged."""
    lens, qlens = [70, 33], [2, 10]
    q, pools, tables = build(lens, qlens, 4, 4, 64, torch.float16, seed=10)
    t, n, cu = dev(tables, lens, qlens)
    out = torch.full((12, 4, 64), 7.0, dtype=torch.float16, device=DEV)
    pa.paged_cross_attention(q.to(DEV), pools[0].to(DEV), pools[1].to(DEV), t, n, 0.125, max_enc_len=70, cu_q_lens=cu,
                             max_q_len=max_q, out=out)
    torch.cuda.synchronize()
    assert pa.device_error() == SEQ_LEN
    check(out[:2], q[:2], pools, tables, lens[:1], [2], 0.125)
    assert bool((out[2:] == 7).all())


@pytest.mark.parametrize("cu", [[0, 3, 99], [0, -4, 5], [5, 3, 12], [-2, 3, 5]])
def test_rows_outside_q_are_neither_read_nor_written(cu):
    lens, qlens = [70, 33], [3, 2]
    q, pools, tables = build(lens, [3, 9], 4, 4, 64, torch.float16, seed=11)
    t, n, _ = dev(tables, lens, qlens)
    c = torch.tensor(cu, dtype=torch.int32, device=DEV)
    for max_q in (8, 99):
        out = torch.full((12, 4, 64), 7.0, dtype=torch.float16, device=DEV)
        pa.paged_cross_attention(q.to(DEV), pools[0].to(DEV), pools[1].to(DEV), t, n, 0.125, max_enc_len=70,
                                 cu_q_lens=c, max_q_len=max_q, out=out)
        torch.cuda.synchronize()
        assert pa.device_error() & SEQ_LEN


def test_no_rows_no_sequences():
    k = torch.zeros(4, 16, 2, 64, dtype=torch.float16, device=DEV)
    q = torch.empty(0, 4, 64, dtype=torch.float16, device=DEV)
    t = torch.zeros(3, 2, dtype=torch.int32, device=DEV)
    n = torch.tensor([5, 0, 2], dtype=torch.int32, device=DEV)
    assert pa.paged_cross_attention(q, k, k, t, n, 1.0).shape == (0, 4, 64)
    cu = torch.zeros(4, dtype=torch.int32, device=DEV)
    assert pa.paged_cross_attention(q, k, k, t, n, 1.0, cu_q_lens=cu).shape == (0, 4, 64)
    assert pa.paged_cross_attention(q, k, k, t[:0], n[:0], 1.0, cu_q_lens=cu[:1]).shape == (0, 4, 64)
    assert pa.device_error() == 0


@pytest.mark.parametrize("qlens", [[4, 4, 4], [1, 30, 4]])
def test_captured_on_a_given_stream(qlens):
    """Replays see new queries, lengths and states; a call on another stream in
    between shares nothing with them."""
    lens = [500, 64, 130]
    q, pools, tables = build(lens, qlens, 8, 2, 64, torch.float16, seed=12)
    t, n, cu = dev(tables, lens, qlens)
    qd, kd, vd = q.to(DEV), pools[0].to(DEV), pools[1].to(DEV)
    out = torch.empty_like(qd)
    ws = torch.empty(max(256, pa.cross_workspace_bytes(3, q.shape[0], max(qlens))), dtype=torch.uint8, device=DEV)

    def call(**kw):
        return pa.paged_cross_attention(qd, kd, vd, t, n, 0.125, max_enc_len=500, cu_q_lens=cu, max_q_len=max(qlens),
                                        **kw)
    call(out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out=out, workspace=ws)
    side = torch.cuda.Stream()
    for lens2 in ([500, 64, 130], [3, 0, 129]):
        n.copy_(torch.tensor(lens2, dtype=torch.int32))
        side.wait_stream(torch.cuda.current_stream())
        other = call(stream=side)
        graph.replay()
        torch.cuda.synchronize()
        check(out, q, pools, tables, lens2, qlens, 0.125)
        assert torch.equal(other, out)
    assert pa.device_error() == 0


def test_two_graphs_share_a_workspace():
    lens, qlens = [100, 40], [20, 9]
    q, pools, tables = build(lens, qlens, 4, 2, 64, torch.float16, seed=13)
    t, n, cu = dev(tables, lens, qlens)
    qd, kd, vd = q.to(DEV), pools[0].to(DEV), pools[1].to(DEV)
    ws = torch.empty(pa.cross_workspace_bytes(2, 29, 20), dtype=torch.uint8, device=DEV)
    outs = [torch.empty_like(qd) for _ in range(2)]
    qs = [qd, qd.flip(0).contiguous()]
    pa.paged_cross_attention(qd, kd, vd, t, n, 0.125, 100, cu, 20, workspace=ws)
    torch.cuda.synchronize()
    graphs = []
    for a, o in zip(qs, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pa.paged_cross_attention(a, kd, vd, t, n, 0.125, 100, cu, 20, out=o, workspace=ws)
        graphs.append(g)
    for _ in range(5):
        graphs[0].replay()
        graphs[1].replay()
    torch.cuda.synchronize()
    check(outs[0], q, pools, tables, lens, qlens, 0.125)
    check(outs[1], q.flip(0), pools, tables, lens, qlens, 0.125)


def test_same_results_every_time():
    lens, qlens = [1500, 700, 20], [5, 40, 1]
    q, pools, tables = build(lens, qlens, 12, 12, 64, torch.bfloat16, seed=14)
    first = run(q, pools, tables, lens, qlens, 0.125)
    for _ in range(10):
        assert torch.equal(run(q, pools, tables, lens, qlens, 0.125), first)


def test_single_rows_agree_with_decode():
    """One row a sequence is what decode computes over the same cache."""
    lens = [5, 512, 1300, 77]
    q, pools, tables = build(lens, [1] * 4, 8, 4, 128, torch.float16, seed=15)
    out = run(q, pools, tables, lens, [1] * 4, 0.09, uniform=True)
    t, n, _ = dev(tables, lens, [1] * 4)
    dec = pa.paged_attention_decode(q.to(DEV), pools[0].to(DEV), pools[1].to(DEV), t, n, 0.09, 1300)
    check(out, q, pools, tables, lens, [1] * 4, 0.09)
    check(dec, q, pools, tables, lens, [1] * 4, 0.09)


@pytest.mark.parametrize("D", [64, 128])
def test_many_sequences_in_order_of_length(D):
    """More items than run at once, which CTAs take longest first: equal lengths,
    none, and lengths that are refused (the lowest number among them)."""
    lens = [int(x) for x in np.random.default_rng(16).integers(0, 90, 50)]
    lens[3] = lens[4] = lens[20] = 33
    qlens = [1 + i % 3 for i in range(50)]
    q, pools, tables = build(lens, qlens, 8, 8, D, torch.float16, seed=16)
    t, n, cu = dev(tables, lens, qlens)
    bad = {0: -2 ** 31, 7: -1, 8: -7, 49: 2 ** 31 - 1, 30: 10 ** 6}
    for b, v in bad.items():
        n[b] = v
    out = pa.paged_cross_attention(q.to(DEV), pools[0].to(DEV), pools[1].to(DEV), t, n, 0.125, max_enc_len=90,
                                   cu_q_lens=cu, max_q_len=3)
    torch.cuda.synchronize()
    assert pa.device_error() == SEQ_LEN
    check(out, q, pools, tables, [0 if b in bad else x for b, x in enumerate(lens)], qlens, 0.125)


def test_two_streams_at_once():
    """Calls on two streams, with chunks and without, share nothing."""
    cases = []
    for seed, qlens in ((17, [4] * 30), (18, [1, 40, 3] * 10)):
        lens = [int(x) for x in np.random.default_rng(seed).integers(0, 300, 30)]
        q, pools, tables = build(lens, qlens, 8, 2, 64, torch.float16, seed=seed)
        cases.append((q, pools, tables, lens, qlens, dev(tables, lens, qlens), q.to(DEV), pools[0].to(DEV), pools[1].to(DEV)))
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in cases], [[], []]
    for _ in range(8):
        for i, (s, c) in enumerate(zip(streams, cases)):
            t, n, cu = c[5]
            outs[i].append(pa.paged_cross_attention(c[6], c[7], c[8], t, n, 0.125, max_enc_len=300, cu_q_lens=cu,
                                                    max_q_len=max(c[4]), stream=s))
    torch.cuda.synchronize()
    for c, got in zip(cases, outs):
        check(got[0], *c[:5], 0.125)
        assert all(torch.equal(g, got[0]) for g in got)
    assert pa.device_error() == 0


@pytest.mark.parametrize("low", [False, True])
@pytest.mark.parametrize("Hq,Hkv,chunks", [(8, 8, 20), (8, 8, 160), (64, 64, 3), (64, 64, 19), (16, 1, 170),
                                           (2, 2, 256), (2, 2, 257), (1, 1, 600)])
def test_more_chunks_than_ctas(Hq, Hkv, chunks, low):
    """Items in two rounds and more, up to and past those that are dealt out by
    their work; also with max_q_len below the chunks' lengths."""
    rng = np.random.default_rng(chunks)
    lens = [int(x) for x in rng.integers(0, 400, chunks)]
    qlens = [int(x) for x in rng.integers(9, 30 if Hkv > 1 else 90, chunks)]
    q, pools, tables = build(lens, qlens, Hq, Hkv, 64, torch.float16, seed=chunks)
    t, n, cu = dev(tables, lens, qlens)
    out = pa.paged_cross_attention(q.to(DEV), pools[0].to(DEV), pools[1].to(DEV), t, n, 0.125, max_enc_len=400,
                                   cu_q_lens=cu, max_q_len=9 if low else max(qlens))
    torch.cuda.synchronize()
    assert pa.device_error() == 0
    check(out, q, pools, tables, lens, qlens, 0.125)
