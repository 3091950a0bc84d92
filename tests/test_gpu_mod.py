"""Attention with capped, distance-biased and windowed scores against a 64-bit
reference: decode, verify rows and prefill chunks over a 16-bit cache."""
import math

import numpy as np
import pytest
import torch

import paged_kv_attention_decode_gb300 as pa
from tests import _ref64 as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def slopes_of(Hq):
    return (2.0 ** (-8.0 * np.arange(1, Hq + 1) / Hq)).astype(np.float32)


MODS = {
    "cap": dict(softcap=20.0),
    "small_cap": dict(softcap=0.5),
    "alibi": dict(alibi=True),
    "window1": dict(window=1),
    "window17": dict(window=17),
    "window200": dict(window=200),
    "wide": dict(window=10 ** 6, softcap=1000.0),
    "all": dict(softcap=30.0, window=150, alibi=True),
    "none": dict(),
}


def build(lens, qlens, Hq, Hkv, D, dt, seed, window=0, qscale=3.0):
    """Scattered blocks; every slot that no query of the step may see (tails,
    unused blocks, keys before the windows) is NaN, and the table entries of
    blocks before the windows are garbage."""
    rng = np.random.default_rng(seed)
    used = [(int(n) + 15) // 16 for n in lens]
    NB = sum(used) + 3
    perm = rng.permutation(NB)
    tables = rng.integers(-9, NB + 9, (len(lens), max(1, max(used))))
    live = np.zeros((NB, 16), bool)
    at = 0
    for b, u in enumerate(used):
        n, c = int(lens[b]), int(qlens[b])
        lo = max(0, n - c + 1 - window) if window else 0
        first = lo // 16
        tables[b, first:u] = perm[at + first:at + u]
        for j in range(lo, n):
            live[perm[at + j // 16], j % 16] = True
        at += u
    g = torch.Generator().manual_seed(seed)
    pools = []
    for _ in range(2):
        x = torch.randn(NB, 16, Hkv, D, generator=g).to(dt)
        x[torch.from_numpy(~live)] = float("nan")
        pools.append(x)
    q = (torch.randn(int(sum(qlens)), Hq, D, generator=g) * qscale).to(dt)
    return q, pools, tables.astype(np.int32)


def run(q, pools, tables, lens, qlens, scale, decode, softcap=0.0, window=0, alibi=False, **kw):
    Hq = q.shape[1]
    sl = torch.from_numpy(slopes_of(Hq)).to(DEV) if alibi else None
    qd, kd, vd = q.to(DEV), pools[0].to(DEV), pools[1].to(DEV)
    td, ld = torch.from_numpy(tables).to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    if decode:
        out = pa.paged_attention_decode_mod(qd, kd, vd, td, ld, scale, int(max(lens)), softcap=softcap, window=window,
                                            alibi_slopes=sl, **kw)
    else:
        cu = torch.tensor(np.concatenate([[0], np.cumsum(qlens)]), dtype=torch.int32, device=DEV)
        out = pa.paged_attention_prefill_mod(qd, kd, vd, td, ld, cu, scale, int(max(qlens)), int(max(lens)),
                                             softcap=softcap, window=window, alibi_slopes=sl, **kw)
    torch.cuda.synchronize()
    return out


def check(out, q, pools, tables, lens, qlens, scale, softcap=0.0, window=0, alibi=False):
    kv = [np.nan_to_num(p.double().numpy()) for p in pools]
    sl = slopes_of(q.shape[1]).astype(np.float64) if alibi else None
    ref, A, smax, cnt = R.attention(q.double().numpy(), *kv, tables, lens, qlens, scale, softcap, window, sl)
    far = float(max(lens)) if alibi else 0.0
    tol = R.bound(ref, A, smax, cnt, max(float(np.abs(kv[1]).max()), 1.0), q.dtype, q.dtype, softcap, far)
    got = out.double().cpu().numpy()
    assert np.all(np.isfinite(got))
    worst = np.max(np.abs(got - ref) / tol) if got.size else 0
    assert worst <= 1, worst


LENS = [1, 2, 16, 17, 33, 100, 511, 512, 513, 1025, 700]


@pytest.mark.parametrize("mod", MODS)
@pytest.mark.parametrize("Hq,Hkv,D,dn", [(4, 4, 128, "f16"), (3, 3, 64, "bf16"), (8, 2, 128, "bf16"),
                                         (16, 1, 64, "f16"), (40, 2, 128, "bf16")])
def test_decode(mod, Hq, Hkv, D, dn):
    m = MODS[mod]
    one = [1] * len(LENS)
    q, pools, tables = build(LENS, one, Hq, Hkv, D, DT[dn], seed=Hq, window=m.get("window", 0))
    out = run(q, pools, tables, LENS, one, 1 / math.sqrt(D), True, **m)
    check(out, q, pools, tables, LENS, one, 1 / math.sqrt(D), **m)
    assert pa.device_error() == 0


@pytest.mark.parametrize("part", [16, 48, 512])
@pytest.mark.parametrize("mod", ["window17", "all"])
def test_decode_partitions(mod, part):
    m = MODS[mod]
    one = [1] * len(LENS)
    for Hq, Hkv in ((2, 2), (8, 2)):
        q, pools, tables = build(LENS, one, Hq, Hkv, 64, torch.float16, seed=part, window=m.get("window", 0))
        out = run(q, pools, tables, LENS, one, 0.125, True, partition_size=part, **m)
        check(out, q, pools, tables, LENS, one, 0.125, **m)
    assert pa.device_error() == 0


@pytest.mark.parametrize("mod", MODS)
@pytest.mark.parametrize("Hq,Hkv,D,dn", [(4, 4, 128, "bf16"), (8, 2, 64, "f16"), (24, 2, 128, "f16")])
def test_verify_and_decode_rows(mod, Hq, Hkv, D, dn):
    m = MODS[mod]
    lens, qlens = [5, 17, 600, 1024, 33, 2, 1300, 8], [5, 8, 3, 1, 2, 2, 7, 8]
    q, pools, tables = build(lens, qlens, Hq, Hkv, D, DT[dn], seed=D, window=m.get("window", 0))
    out = run(q, pools, tables, lens, qlens, 1 / math.sqrt(D), False, **m)
    check(out, q, pools, tables, lens, qlens, 1 / math.sqrt(D), **m)
    assert pa.device_error() == 0


def test_verify_columns_whose_window_starts_in_a_later_partition():
    # 8 queries of 8 heads: four chunks of 16 columns; with partitions of 512
    # and a window that starts near 512 some chunks see nothing of the first one
    for n in (517, 519, 523, 600):
        m = dict(window=n - 513)
        lens, qlens = [n, 40], [8, 1]
        q, pools, tables = build(lens, qlens, 8, 1, 128, torch.bfloat16, seed=n, window=m["window"])
        out = run(q, pools, tables, lens, qlens, 0.09, False, **m)
        check(out, q, pools, tables, lens, qlens, 0.09, **m)
        assert pa.device_error() == 0


STEP = [(300, 300), (500, 37), (213, 9), (400, 150), (50, 2), (700, 8), (90, 4), (549, 1), (16, 1), (1, 1), (129, 128),
        (900, 300)]


@pytest.mark.parametrize("mod", MODS)
@pytest.mark.parametrize("Hq,Hkv,D,dn", [(4, 4, 128, "f16"), (8, 2, 128, "bf16"), (6, 2, 64, "bf16"),
                                         (16, 1, 64, "f16")])
def test_varlen_step(mod, Hq, Hkv, D, dn):
    m = MODS[mod]
    lens, qlens = zip(*STEP)
    q, pools, tables = build(lens, qlens, Hq, Hkv, D, DT[dn], seed=Hq + Hkv, window=m.get("window", 0))
    out = run(q, pools, tables, list(lens), qlens, 1 / math.sqrt(D), False, **m)
    check(out, q, pools, tables, lens, qlens, 1 / math.sqrt(D), **m)
    assert pa.device_error() == 0


def test_chunks_alone_and_negative_scale():
    lens, qlens = [1000, 640], [260, 640]
    for m in (dict(softcap=5.0, window=300), dict(alibi=True)):
        q, pools, tables = build(lens, qlens, 4, 2, 128, torch.bfloat16, seed=1, window=m.get("window", 0))
        out = run(q, pools, tables, lens, qlens, -0.1, False, **m)
        check(out, q, pools, tables, lens, qlens, -0.1, **m)


def test_no_modification_matches_the_plain_calls():
    lens, qlens = zip(*STEP)
    q, pools, tables = build(lens, qlens, 8, 2, 128, torch.bfloat16, seed=3)
    out = run(q, pools, tables, list(lens), qlens, 0.09, False)
    qd, kd, vd = q.to(DEV), pools[0].to(DEV), pools[1].to(DEV)
    td, ld = torch.from_numpy(tables).to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(qlens)]), dtype=torch.int32, device=DEV)
    ref = pa.paged_attention_prefill(qd, kd, vd, td, ld, cu, 0.09, int(max(qlens)), int(max(lens)))
    # both round P and the output alike; the references of the lazy rescale may differ
    assert torch.all((out.float() - ref.float()).abs() <= 2.0 ** -6 * ref.float().abs() + 2.0 ** -6)


@pytest.mark.parametrize("window", [0, 40])
def test_bad_blocks_inside_the_window_are_masked(window):
    lens, qlens = [200, 300, 45], [100, 2, 1]
    q, pools, tables = build(lens, qlens, 4, 2, 64, torch.float16, seed=5, window=window)
    # one visible block of each row outside the pool
    tables[0, 10], tables[1, 18], tables[2, 1] = 10 ** 7, -3, -1
    m = dict(window=window, softcap=10.0)
    out = run(q, pools, tables, lens, qlens, 0.125, False, **m)
    check(out, q, pools, tables, lens, qlens, 0.125, **m)
    assert pa.device_error() == 1


def test_large_window_context():
    lens, qlens = [20000, 9000], [1, 40]
    m = dict(window=4000, softcap=50.0)
    q, pools, tables = build(lens, qlens, 4, 2, 64, torch.bfloat16, seed=6, window=4000)
    out = run(q, pools, tables, lens, qlens, 0.125, False, **m)
    check(out, q, pools, tables, lens, qlens, 0.125, **m)
    assert pa.device_error() == 0


@pytest.mark.parametrize("Hq,Hkv,D,chunks", [
    (32, 8, 64, [(1600, 1536)]),                 # 192 items: 40 in the last round of 152
    (32, 8, 128, [(1000, 640), (640, 640)]),     # 160 items: 8 in the last round
    (10, 2, 64, [(2048, 2048), (900, 41)]),      # tiles of 25 queries of 5 heads; 84 items: one round
    (4, 2, 64, [(5000, 4900), (4900, 4900), (333, 130)]),   # 156 items of two heads, a pair of one tile among them
])
def test_windowed_chunks_of_several_rounds(Hq, Hkv, D, chunks):
    """More work items than SMs: every row is written, and a sample of them
    agrees with one-token calls over the same keys."""
    lens, qlens = zip(*chunks)
    for m in (dict(window=150), dict(window=90, softcap=15.0)):
        q, pools, tables = build(lens, qlens, Hq, Hkv, D, torch.bfloat16, seed=D + Hq, window=m["window"])
        out = torch.full_like(q, float("nan")).to(DEV)
        run(q, pools, tables, list(lens), qlens, 0.1, False, out=out, **m)
        assert torch.all(torch.isfinite(out))
        # a decode call per sampled row (its own kernel) sees the same keys
        rows, at = [], 0
        for b, (n, c) in enumerate(chunks):
            rows += [(b, at + i, n - c + i + 1) for i in range(0, c, 37)]
            rows.append((b, at + c - 1, n))
            at += c
        sel = torch.tensor([r for _, r, _ in rows])
        sl = [n for _, _, n in rows]
        one = run(q[sel], pools, tables[[b for b, _, _ in rows]], sl, [1] * len(rows), 0.1, True, **m)
        got, ref = out[sel.to(DEV)].float(), one.float()
        # each kernel rounds its weights to bf16 (2^-8 of sum p |v| <= 2) and its result (2^-8 of it)
        assert torch.all((got - ref).abs() <= 2.0 ** -6 * ref.abs() + 2.0 ** -6)
        assert pa.device_error() == 0
