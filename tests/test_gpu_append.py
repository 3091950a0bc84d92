"""Rotating and appending new tokens to 16-bit, FP8 and 4-bit caches, and the
4-bit cache's write, unpack and block copy, against 64-bit references.  Codes
are compared bit for bit (the quantisers' definitions fix every fp32 step)."""
import numpy as np
import pytest
import torch

import paged_kv_attention_decode_gb300 as pa
from tests import _ref64 as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def table(rot, n, seed=0):
    half = rot // 2
    ang = np.arange(n)[:, None] * 10000.0 ** (-np.arange(half) / half)
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def tokens(T, Hq, Hkv, D, dt, seed, fused=False):
    g = torch.Generator().manual_seed(seed)
    if fused:      # slices of one projection's rows, with a gap behind them
        x = torch.randn(T, (Hq + 2 * Hkv) * D + 24, generator=g).to(dt).to(DEV)
        q = x[:, :Hq * D].unflatten(1, (Hq, D))
        k = x[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
        v = x[:, (Hq + Hkv) * D:(Hq + 2 * Hkv) * D].unflatten(1, (Hkv, D))
        return q, k, v
    return tuple(torch.randn(T, h, D, generator=g).to(dt).to(DEV) for h in (Hq, Hkv, Hkv))


def slots_for(T, NB, seed):
    s = np.random.default_rng(seed).permutation(NB * 16)[:T].astype(np.int64)
    if T > 4:
        s[3] = -1
    return s


def np32(t):
    return t.detach().float().cpu().numpy()


def bits16(t):
    return t.detach().contiguous().cpu().view(torch.int16).numpy()


CASES = [
    # T, Hq, Hkv, D, rot, interleaved, dtype, fused
    (1, 8, 2, 128, 128, False, "bf16", False),
    (1, 1, 1, 64, 16, True, "f16", False),
    (17, 32, 8, 128, 128, False, "f16", True),
    (33, 6, 3, 64, 64, False, "bf16", True),
    (130, 12, 4, 128, 64, True, "bf16", True),
    (7, 5, 5, 128, 48, False, "f16", False),
    (65, 3, 1, 64, 48, True, "bf16", False),
    (1500, 4, 2, 128, 80, False, "bf16", True),
    (40, 0, 3, 128, 128, False, "bf16", False),     # keys and values alone
]


def rope_case(case, cache):
    T, Hq, Hkv, D, rot, inter, dn, fused = case
    dt = DT[dn]
    q, k, v = tokens(T, Hq, Hkv, D, dt, seed=T + D, fused=fused)
    NB = (T + 15) // 16 + 3
    slots = slots_for(T, NB, T)
    npos = 4096
    pos = np.random.default_rng(T + 1).integers(0, npos, T).astype(np.int64)
    pos[0] = npos - 1
    cs = table(rot, npos)
    dev = [torch.from_numpy(a).to(DEV) for a in (slots, pos, cs)]
    return T, Hq, Hkv, D, rot, inter, dt, q, k, v, NB, slots, pos, cs, dev


def check_q(q_out, q, cs, pos, rot, inter, dt):
    ref, mag = R.rope64(np32(q), cs, pos, rot, inter)
    # two products and a sum in fp32 (2^-24 of each), then one rounding to dt
    tol = 2.0 ** -22 * mag + R.U[dt] * np.abs(ref) * (1 + 2.0 ** -8) + R.SUB[dt]
    assert np.all(np.abs(np32(q_out).astype(np.float64) - ref) <= tol)
    step = torch.from_numpy(R.rope32(np32(q), cs, pos, rot, inter)).to(dt)
    assert np.array_equal(bits16(q_out), bits16(step))     # the definition's fp32 steps, bit for bit


@pytest.mark.parametrize("case", CASES)
def test_rope_append_16bit(case):
    T, Hq, Hkv, D, rot, inter, dt, q, k, v, NB, slots, pos, cs, (sl, ps, tb) = rope_case(case, "same")
    kc, vc = (torch.randn(NB, 16, Hkv, D).to(dt).to(DEV) for _ in range(2))
    want_k, want_v = bits16(kc).reshape(NB * 16, Hkv, D).copy(), bits16(vc).reshape(NB * 16, Hkv, D).copy()
    before = [bits16(x) for x in (q, k, v)]
    out = pa.paged_rope_kv_write(q, k, v, kc, vc, sl, ps, tb, interleaved=inter)
    torch.cuda.synchronize()
    check_q(out, q, cs, pos, rot, inter, dt)
    live = slots >= 0
    step = torch.from_numpy(R.rope32(np32(k), cs, pos, rot, inter)).to(dt)
    want_k[slots[live]] = bits16(step)[live]
    want_v[slots[live]] = bits16(v)[live]
    assert np.array_equal(bits16(kc).reshape(want_k.shape), want_k)
    assert np.array_equal(bits16(vc).reshape(want_v.shape), want_v)
    for x, b in zip((q, k, v), before):
        assert np.array_equal(bits16(x), b)                # the inputs stay
    assert pa.device_error() == 0


@pytest.mark.parametrize("case", [c for c in CASES if c[3] == 128])
@pytest.mark.parametrize("scale", [1 / 16, 0.013])
def test_rope_append_fp8(case, scale):
    T, Hq, Hkv, D, rot, inter, dt, q, k, v, NB, slots, pos, cs, (sl, ps, tb) = rope_case(case, "fp8")
    kc, vc = (torch.randint(0, 256, (NB, Hkv, 16, D), dtype=torch.uint8).to(DEV) for _ in range(2))
    want = [x.cpu().numpy().copy() for x in (kc, vc)]
    out = pa.paged_rope_kv_write_fp8(q, k, v, kc, vc, sl, ps, tb, scale, scale, interleaved=inter)
    torch.cuda.synchronize()
    check_q(out, q, cs, pos, rot, inter, dt)
    inv = np.float32(1.0) / np.float32(scale)
    for x, w, got in ((R.rope32(np32(k), cs, pos, rot, inter), want[0], kc), (np32(v), want[1], vc)):
        y = (x * inv).astype(np.float32)
        mag = R.nearest_even(np.abs(y).astype(np.float64), R.E4M3[:127])
        codes = (mag | (np.signbit(y) << 7)).astype(np.uint8)
        live = slots >= 0
        w[slots[live] // 16, :, slots[live] % 16] = codes[live]
        assert np.array_equal(got.cpu().numpy(), w)
    assert pa.device_error() == 0


def fp4_pools(NB, Hkv, D, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randint(0, 256, (NB, Hkv, pa.fp4_tile_bytes(D)), dtype=torch.uint8, generator=g).to(DEV)
            for _ in range(2)]


def check_fp4(pools, before, rows, slots, scale):
    live = slots >= 0
    for got, old, x, isv in zip(pools, before, rows, (False, True)):
        codes, sc = (a.copy() for a in R.unpack_tiles(old, isv))
        c, s = R.quantise_fp4(x[live], scale)
        blk, off = slots[live] // 16, slots[live] % 16
        codes[blk, off], sc[blk, off] = c, s
        want = R.pack_tiles(codes, sc, isv)
        assert np.array_equal(got.cpu().numpy(), want)     # every byte, the untouched slots too


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("scale", [1 / 256, 0.0031])
def test_rope_append_fp4(case, scale):
    T, Hq, Hkv, D, rot, inter, dt, q, k, v, NB, slots, pos, cs, (sl, ps, tb) = rope_case(case, "fp4")
    pools = fp4_pools(NB, Hkv, D, T)
    before = [x.cpu().numpy().copy() for x in pools]
    out = pa.paged_rope_kv_write_fp4(q, k, v, *pools, sl, ps, tb, scale, scale, interleaved=inter)
    torch.cuda.synchronize()
    check_q(out, q, cs, pos, rot, inter, dt)
    check_fp4(pools, before, (R.rope32(np32(k), cs, pos, rot, inter), np32(v)), slots, scale)
    assert pa.device_error() == 0


@pytest.mark.parametrize("T,Hkv,D,dn,scale", [(1, 1, 64, "f16", 1.0), (19, 8, 128, "bf16", 1 / 256),
                                              (300, 3, 64, "bf16", 0.01), (77, 32, 128, "f16", 1 / 64)])
def test_write_fp4_and_unpack(T, Hkv, D, dn, scale):
    dt = DT[dn]
    _, k, v = tokens(T, 1, Hkv, D, dt, seed=T)
    k[0] *= 1e-6                      # scales that round to 0
    if T > 2:
        k[1, 0, :16] = 0
        k[2] *= 3000.0                # saturating scales (fp16: up to infinity)
        v[1, :, 5] = float("nan")     # a NaN group
        v[2, 0, 0] = float("inf")
    # values on the rounding borders of the codes and of the scales
    v[0, 0, :16] = torch.tensor([6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -5, -3.5, -2.5, -0.25, 0, -0.0, 4.999, 0.2501])
    NB = (T + 15) // 16 + 2
    slots = slots_for(T, NB, T)
    pools = fp4_pools(NB, Hkv, D, 1)
    before = [x.cpu().numpy().copy() for x in pools]
    pa.paged_kv_write_fp4(k, v, *pools, torch.from_numpy(slots).to(DEV), scale, scale)
    torch.cuda.synchronize()
    check_fp4(pools, before, (np32(k), np32(v)), slots, scale)
    for out, pool, isv in zip(pa.paged_kv_unpack_fp4(*pools, scale, scale, dt), pools, (False, True)):
        ref = R.tile_values(pool.cpu().numpy(), isv, float(np.float32(scale)))
        got = np32(out).astype(np.float64)
        nan = np.isnan(ref)
        assert np.array_equal(np.isnan(got), nan)
        big = 65504.0 if dt == torch.float16 else 3e38
        fin = ~nan & (np.abs(ref) < big)
        tol = (R.U[dt] + 2.0 ** -23) * np.abs(ref) + R.SUB[dt]
        assert np.all(np.abs(got - ref)[fin] <= tol[fin])
    assert pa.device_error() == 0


@pytest.mark.parametrize("inter", [False, True])
def test_query_rotated_in_place(inter):
    dt = torch.bfloat16
    q, k, v = tokens(50, 8, 2, 128, dt, seed=3, fused=True)
    rot, cs = 96, table(96, 512)
    pos = np.arange(50, dtype=np.int64) * 10
    slots = torch.arange(50, dtype=torch.int64, device=DEV)
    kc, vc = (torch.zeros(4, 16, 2, 128, dtype=dt, device=DEV) for _ in range(2))
    src, kv = q.clone(), (bits16(k), bits16(v))
    out = pa.paged_rope_kv_write(q, k, v, kc, vc, slots, torch.from_numpy(pos).to(DEV), torch.from_numpy(cs).to(DEV),
                                 interleaved=inter, q_out=q)
    torch.cuda.synchronize()
    assert out is q
    check_q(q, src, cs, pos, rot, inter, dt)
    assert np.array_equal(bits16(k), kv[0]) and np.array_equal(bits16(v), kv[1])


@pytest.mark.parametrize("cache", ["same", "fp8", "fp4"])
def test_bad_rows_are_dropped_and_flagged(cache):
    dt, T, D = torch.bfloat16, 9, 128
    q, k, v = tokens(T, 4, 2, D, dt, seed=5)
    cs = torch.from_numpy(table(D, 100)).to(DEV)
    good = torch.arange(T, dtype=torch.int64, device=DEV)

    def call(slots, pos):
        out = torch.full_like(q, 7.0)
        if cache == "same":
            pools = [torch.zeros(2, 16, 2, D, dtype=dt, device=DEV) for _ in range(2)]
            pa.paged_rope_kv_write(q, k, v, *pools, slots, pos, cs, q_out=out)
        elif cache == "fp8":
            pools = [torch.zeros(2, 2, 16, D, dtype=torch.uint8, device=DEV) for _ in range(2)]
            pa.paged_rope_kv_write_fp8(q, k, v, *pools, slots, pos, cs, 0.1, 0.1, q_out=out)
        else:
            pools = [torch.zeros(2, 2, 9 * D, dtype=torch.uint8, device=DEV) for _ in range(2)]
            pa.paged_rope_kv_write_fp4(q, k, v, *pools, slots, pos, cs, 0.01, 0.01, q_out=out)
        return out, pools, pa.device_error()

    ref, full, err = call(good, good)
    assert err == 0
    pos = good.clone()
    pos[2], pos[4] = -1, 100
    out, pools, err = call(good, pos)
    assert err == 32
    keep = [i for i in range(T) if i not in (2, 4)]
    assert torch.equal(out[keep], ref[keep])
    assert torch.all(out[[2, 4]] == 7.0)
    slots = good.clone()
    slots[1], slots[3] = 32, -5          # past the pool; padding
    out, pools, err = call(slots, good)
    assert err == 2
    assert torch.equal(out, ref)         # the query rows are still rotated
    if cache == "same":
        assert torch.all(pools[0][0, [1, 3]] == 0) and torch.equal(pools[0][0, [0, 2, 4]], full[0][0, [0, 2, 4]])


def test_copy_blocks_fp4():
    k, v = fp4_pools(6, 3, 128, 9)
    ref = [x.clone() for x in (k, v)]
    pa.copy_blocks(k, v, torch.tensor([[0, 4], [2, 1]], dtype=torch.int32, device=DEV))
    for x, r in zip((k, v), ref):
        r[4], r[1] = r[0].clone(), r[2].clone()
        assert torch.equal(x, r)


def test_empty_step():
    dt = torch.float16
    q, k, v = (torch.empty(0, h, 64, dtype=dt, device=DEV) for h in (4, 2, 2))
    pools = fp4_pools(2, 2, 64, 1)
    none = torch.empty(0, dtype=torch.int64, device=DEV)
    before = [x.clone() for x in pools]
    pa.paged_kv_write_fp4(k, v, *pools, none, 1.0, 1.0)
    out = pa.paged_rope_kv_write_fp4(q, k, v, *pools, none, none, torch.zeros(4, 64, device=DEV), 1.0, 1.0)
    torch.cuda.synchronize()
    assert out.shape == q.shape and all(torch.equal(a, b) for a, b in zip(pools, before))


@pytest.mark.parametrize("T,Hq,Hkv,D,dn", [(1, 4, 1, 64, "f16"), (23, 6, 2, 64, "bf16"), (600, 12, 4, 128, "f16")])
def test_write_fp4_of_fused_rows(T, Hq, Hkv, D, dn):
    """Rows that are slices of a fused projection (and one side of them dense)."""
    _, k, v = tokens(T, Hq, Hkv, D, DT[dn], seed=T, fused=True)
    NB = (T + 15) // 16 + 2
    slots = slots_for(T, NB, T)
    for a, b in ((k, v), (k, v.contiguous()), (k.contiguous(), v)):
        pools = fp4_pools(NB, Hkv, D, 2)
        before = [x.cpu().numpy().copy() for x in pools]
        pa.paged_kv_write_fp4(a, b, *pools, torch.from_numpy(slots).to(DEV), 1 / 256, 0.003)
        torch.cuda.synchronize()
        for i, (x, scale) in enumerate(((k, 1 / 256), (v, 0.003))):
            live, isv = slots >= 0, bool(i)
            codes, sc = (y.copy() for y in R.unpack_tiles(before[i], isv))
            codes[slots[live] // 16, slots[live] % 16], sc[slots[live] // 16, slots[live] % 16] = \
                R.quantise_fp4(np32(x)[live], scale)
            assert np.array_equal(pools[i].cpu().numpy(), R.pack_tiles(codes, sc, isv))
    assert pa.device_error() == 0
