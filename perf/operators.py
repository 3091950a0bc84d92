"""Cases of the append, 4-bit cache and modified-score attention operators.

Each case is one call (or the short chain of calls) that a serving step makes:
rotating and appending new tokens to a paged cache, attention over a cache
held in 4 bits, and attention whose scores are capped, biased by distance or
limited to a window.  `run` computes a case in plain torch operations, or,
with `own` true, through this package's entry points; `exact` gives the same
outputs from the definitions in 64 bits.
"""
import math
import random

import torch

own = False
DEV = "cuda"
BS = 16
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
# KV scales of the quantised pools: powers of two, as the calibration of a
# cache of unit-variance rows rounds them
KV8_SCALE = 1.0 / 16
KV4_SCALE = 1.0 / 256
FAR = 131072          # positions covered by the rotation table


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _append(name, T, hq, hkv, d, dt, cache, rot, inter=False, fused=False):
    c = {"op": "append", "T": T, "hq": hq, "hkv": hkv, "d": d, "dt": dt, "cache": cache, "rot": rot,
         "inter": inter, "fused": fused}
    return dict(c, name=name) if name else c


def _attn(name, op, seqs, lo, hi, hq, hkv, d, dt, lens_seed, chunks=0, chunk=0, prefix=0, verify=1, softcap=0.0,
          window=0, alibi=False):
    c = {"op": op, "seqs": seqs, "lo": lo, "hi": hi, "hq": hq, "hkv": hkv, "d": d, "dt": dt,
         "lens_seed": lens_seed, "chunks": chunks, "chunk": chunk, "prefix": prefix, "verify": verify,
         "softcap": softcap, "window": window, "alibi": alibi}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one new token of one sequence, grouped heads: the latency of an append
        _append("append_1_token", 1, 32, 8, 128, "bf16", "same", 128),
        # a decode step of 64 sequences into an 8-bit cache
        _append("append_64_fp8", 64, 32, 32, 128, "f16", "fp8", 128),
        # a full token budget of prompt rows, taken from the rows of a fused QKV product
        _append("append_8192_fused", 8192, 32, 8, 128, "bf16", "same", 128, fused=True),
        # a prompt chunk into a 4-bit cache, half of each head rotated, in adjacent pairs
        _append("append_2049_fp4", 2049, 64, 8, 128, "bf16", "fp4", 64, inter=True),
        # rows that were rotated elsewhere, quantised into a 4-bit cache of short heads
        _append("write_513_fp4_d64", 513, 32, 32, 64, "f16", "fp4", 0),
        # a few short sequences: the latency of a 4-bit decode
        _attn("fp4_decode_small", "fp4", 4, 1, 100, 4, 4, 64, "f16", 1),
        # the B=64 decode step of a 32-head model, contexts U[512, 4096]
        _attn("fp4_decode_b64", "fp4", 64, 512, 4096, 32, 32, 128, "f16", 2),
        # eight long contexts, eight query heads per KV head
        _attn("fp4_decode_long", "fp4", 8, 32768, 131072, 64, 8, 128, "bf16", 3),
        # a mixed step: four prompt chunks on cached prefixes beside verify and decode rows
        _attn("fp4_step", "fp4", 60, 256, 4096, 32, 8, 128, "bf16", 4, chunks=4, chunk=1536, prefix=4096, verify=4),
        # a small batch with a distance bias, heads of 64
        _attn("mod_decode_alibi", "mod", 3, 20, 700, 8, 8, 64, "f16", 5, alibi=True),
        # 256 decode rows that see a window of 1024 tokens, capped scores
        _attn("mod_decode_window", "mod", 256, 128, 8192, 32, 8, 128, "bf16", 6, softcap=50.0, window=1024),
        # prompt chunks beside verify rows: a window of 2048 tokens, capped scores
        _attn("mod_step_window_cap", "mod", 12, 256, 4096, 32, 8, 128, "bf16", 7, chunks=4, chunk=1536, prefix=4096,
              verify=3, softcap=30.0, window=2048),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append", "fp4", "fp4", "mod", "mod"])
    hq, hkv = rng.choice([(32, 32), (32, 8), (64, 8), (8, 8), (12, 4), (16, 2), (6, 2), (8, 1)])
    d = rng.choice([64, 128])
    dt = rng.choice(["f16", "bf16"])
    if op == "append":
        cache = rng.choice(["same", "fp8", "fp4"])
        if cache == "fp8":
            d = 128
        rot = rng.choice([d, d, d // 2, 0 if cache == "fp4" else d])
        T = _log(rng, 1, max(1, 8192 * 8 // max(8, hkv)))
        return _append(None, T, hq, hkv, d, dt, cache, rot, rng.random() < 0.4, rng.random() < 0.5)
    seed = rng.randrange(1 << 20)
    extra = {}
    if op == "mod":
        kind = rng.randrange(4)
        extra = {"softcap": rng.choice([15.0, 30.0, 50.0]) if kind in (0, 3) else 0.0,
                 "window": _log(rng, 16, 4096) if kind in (1, 3) else 0, "alibi": kind == 2}
    if rng.random() < 0.6:
        seqs = _log(rng, 1, 64)
        budget = 64 * 4096 * 8 // (seqs * max(8, hkv))   # tokens per sequence that keep the pools in bounds
        hi = _log(rng, 40, max(41, min(131072, budget)))
        return _attn(None, op, seqs, max(1, hi // 16), hi, hq, hkv, d, dt, seed, **extra)
    chunk = _log(rng, 9, 1536)
    return _attn(None, op, _log(rng, 1, 48), 16, _log(rng, 64, 2048), hq, hkv, d, dt, seed,
                 chunks=rng.randint(1, 4), chunk=chunk, prefix=_log(rng, 16, 4096), verify=rng.randint(1, 8), **extra)


def _lens(case):
    """(context length, new tokens) of every sequence: chunks first, then the short rows."""
    rng = random.Random(case["lens_seed"])
    rows = []
    for _ in range(case["chunks"]):
        rows.append((rng.randint(0, case["prefix"]) + case["chunk"], case["chunk"]))
    for i in range(case["seqs"]):
        n = rng.randint(case["lo"], case["hi"])
        rows.append((n, min(n, 1 + i % case["verify"])))
    return rows


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(g, *shape, dt=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).to(dt)


def _e2m1(y):
    """Nearest E2M1 magnitude codes (ties to even) of |y|, sign in bit 3."""
    a = y.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return code.to(torch.uint8) | (torch.signbit(y).to(torch.uint8) << 3)


def _quantise4(x, scale):
    """Rows [..., D] in fp32 -> (codes [..., D] uint8, E4M3 group scales [..., D / 16])."""
    y = x * (1.0 / scale)
    grp = y.unflatten(-1, (-1, 16))
    six = torch.full((1,), 6.0, device=x.device)         # a tensor: a division, not a product with 1 / 6
    s8 = (grp.abs().amax(-1) / six).clamp(max=448.0).to(torch.float8_e4m3fn)
    sv = s8.float().unsqueeze(-1)
    q = torch.where(sv > 0, grp / torch.where(sv > 0, sv, six), torch.zeros_like(grp))
    return _e2m1(q).flatten(-2), s8.view(torch.uint8)


def _tiles(codes, scales, v):
    """Head-major tiles [NB, H, bytes] from token-major blocks: codes
    [NB, 16, H, D] and scales [NB, 16, H, D / 16].  A tile holds 16 rows of
    D / 2 code bytes (even dimension in the low nibble), then the scales:
    token-major for K, group-major for V."""
    c = (codes[..., 0::2] | (codes[..., 1::2] << 4)).permute(0, 2, 1, 3).flatten(2)
    s = scales.permute(0, 2, 3, 1) if v else scales.permute(0, 2, 1, 3)
    return torch.cat([c, s.flatten(2)], -1).contiguous()


def _prepare_append(case, seed):
    g = _gen(seed)
    T, hq, hkv, d, dt = case["T"], case["hq"], case["hkv"], case["d"], TYPES[case["dt"]]
    if case["fused"]:
        qkv = _randn(g, T, (hq + 2 * hkv) * d, dt=dt)
        q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([hq * d, hkv * d, hkv * d], 1))
    else:
        q, k, v = _randn(g, T, hq, d, dt=dt), _randn(g, T, hkv, d, dt=dt), _randn(g, T, hkv, d, dt=dt)
    nb = (T + BS - 1) // BS + 4
    slots = torch.randperm(nb * BS, generator=g, device=DEV)[:T].contiguous()
    if T > 16:       # runs of consecutive slots, as a prompt's blocks are filled
        blocks = torch.randperm(nb, generator=g, device=DEV)
        i = torch.arange(T, device=DEV)
        slots = blocks[i // BS] * BS + i % BS
        slots[T // 2] = -1                                     # a padding row
    st = {"q": q, "k": k, "v": v, "slots": slots, "pos": None, "table": None}
    if case["rot"]:
        half = case["rot"] // 2
        freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=DEV) / half)
        ang = torch.arange(FAR, dtype=torch.float64, device=DEV)[:, None] * freq
        st["table"] = torch.cat([ang.cos(), ang.sin()], 1).float()
        start = int(torch.randint(0, FAR - T, (1,), generator=g, device=DEV))
        st["pos"] = torch.arange(start, start + T, device=DEV)
    if case["cache"] == "same":
        st["pools"] = [_randn(g, nb, BS, hkv, d, dt=dt) for _ in range(2)]
    elif case["cache"] == "fp8":
        st["pools"] = [(_randn(g, nb, hkv, BS, d) / KV8_SCALE).clamp(-448, 448).to(torch.float8_e4m3fn)
                       .view(torch.uint8) for _ in range(2)]
    else:
        st["pools"] = [_tiles(*_quantise4(_randn(g, nb, BS, hkv, d), KV4_SCALE), v) for v in (False, True)]
    return st


def _prepare_attn(case, seed):
    g = _gen(seed)
    rows = _lens(case)
    hq, hkv, d, dt = case["hq"], case["hkv"], case["d"], TYPES[case["dt"]]
    n = torch.tensor([r[0] for r in rows], dtype=torch.int32)
    ql = torch.tensor([r[1] for r in rows], dtype=torch.int32)
    used = [(r[0] + BS - 1) // BS for r in rows]
    nb = int(sum(used) * 1.1) + 4
    perm = torch.randperm(nb, generator=g, device=DEV).to(torch.int32)
    tables = torch.zeros(len(rows), max(used), dtype=torch.int32, device=DEV)
    at = 0
    for b, u in enumerate(used):
        tables[b, :u] = perm[at:at + u]
        at += u
    cu = torch.zeros(len(rows) + 1, dtype=torch.int32)
    cu[1:] = ql.cumsum(0)
    st = {"q": _randn(g, int(cu[-1]), hq, d, dt=dt), "tables": tables, "lens": n.to(DEV), "cu": cu.to(DEV),
          "rows": rows, "scale": 1.0 / math.sqrt(d), "slopes": None, "max_len": int(n.max()),
          "chunk_kv": sum(r[0] for r in rows if r[1] > 8)}
    if case["softcap"]:
        st["q"] = st["q"] * 4        # scores that reach the cap's bend
    if case["alibi"]:
        st["slopes"] = 2.0 ** (-8.0 * torch.arange(1, hq + 1, device=DEV, dtype=torch.float32) / hq)
    pools = []
    for v in (False, True):
        if case["op"] == "fp4":
            pool = torch.empty(nb, hkv, BS * d // 2 + d, dtype=torch.uint8, device=DEV)
            step = max(1, (1 << 26) // (BS * hkv * d))
            for b0 in range(0, nb, step):
                b1 = min(nb, b0 + step)
                pool[b0:b1] = _tiles(*_quantise4(_randn(g, b1 - b0, BS, hkv, d), KV4_SCALE), v)
        else:
            pool = torch.empty(nb, BS, hkv, d, dtype=dt, device=DEV)
            step = max(1, (1 << 27) // (BS * hkv * d))
            for b0 in range(0, nb, step):
                b1 = min(nb, b0 + step)
                pool[b0:b1] = _randn(g, b1 - b0, BS, hkv, d)
        pools.append(pool)
    st["pools"] = pools
    return st


def prepare(case, seed):
    st = _prepare_append(case, seed) if case["op"] == "append" else _prepare_attn(case, seed)
    st["case"] = case
    return st


# ---------------------------------------------------------------------------
# plain forms: 32 bits, rounded once at the end
# ---------------------------------------------------------------------------
def _rotate(x, cs, rot, inter):
    """Rows [T, H, D] in fp32, cos and sin [T, rot] of their positions."""
    c, s = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])
    a, b = a * c - b * s, b * c + a * s
    y = torch.stack([a, b], -1).flatten(-2) if inter else torch.cat([a, b], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _values4(tiles, d, v):
    """Code times group scale of head-major tiles [..., H, bytes] -> fp32 [..., H, 16, D]."""
    n = BS * d // 2
    mags = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=tiles.device)
    lut = torch.cat([mags, -mags])
    both = torch.stack([lut[torch.arange(256, device=tiles.device) & 15], lut[torch.arange(256, device=tiles.device) >> 4]], 1)
    x = both[tiles[..., :n].int()].unflatten(-2, (BS, d // 2)).flatten(-2)
    s = tiles[..., n:].contiguous().view(torch.float8_e4m3fn).float()
    s = s.unflatten(-1, (d // 16, BS)).transpose(-1, -2) if v else s.unflatten(-1, (BS, d // 16))
    return (x.unflatten(-1, (d // 16, 16)) * s.unsqueeze(-1)).flatten(-2)


def _plain_append(st):
    case = st["case"]
    q, k, v = st["q"].float(), st["k"].float(), st["v"].float()
    if case["rot"]:
        cs = st["table"][st["pos"]]
        q, k = _rotate(q, cs, case["rot"], case["inter"]), _rotate(k, cs, case["rot"], case["inter"])
    q = q.to(st["q"].dtype)
    live = st["slots"] >= 0
    blk, off = (st["slots"] // BS)[live], (st["slots"] % BS)[live]
    got = []
    for x, pool, isv in ((k, st["pools"][0], False), (v, st["pools"][1], True)):
        x = x[live]
        if case["cache"] == "same":
            pool[blk, off] = x.to(pool.dtype)
            got.append(pool)
        elif case["cache"] == "fp8":
            pool[blk, :, off] = (x * (1.0 / KV8_SCALE)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            got.append(pool.view(torch.float8_e4m3fn))
        else:
            d, half = case["d"], case["d"] // 2
            codes, s = _quantise4(x, KV4_SCALE)
            body = pool[..., :BS * half].unflatten(-1, (BS, half))
            body[blk, :, off] = codes[..., 0::2] | (codes[..., 1::2] << 4)
            tail = pool[..., BS * half:]
            if isv:
                tail.unflatten(-1, (d // 16, BS))[blk, :, :, off] = s
            else:
                tail.unflatten(-1, (BS, d // 16))[blk, :, off] = s
            got.append((_values4(pool, d, isv) * KV4_SCALE).transpose(1, 2).to(q.dtype))
    return [q, *got] if case["rot"] else got


def _plain_group(st, b0, b1, dst):
    """Attention of sequences b0..b1-1, padded to their longest context and chunk."""
    case, rows = st["case"], st["rows"][b0:b1]
    if not rows:
        return
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    B, N, Q = len(rows), max(r[0] for r in rows), max(r[1] for r in rows)
    nblk = (N + BS - 1) // BS
    tab = st["tables"][b0:b1, :nblk].long()
    lens, first = st["lens"][b0:b1].long(), st["cu"][b0:b1].long()
    ql = st["cu"][b0 + 1:b1 + 1].long() - first
    kv = []
    for pool, isv in zip(st["pools"], (False, True)):
        x = pool[tab]
        if case["op"] == "fp4":
            x = _values4(x, d, isv).transpose(1, 2).flatten(2, 3) * KV4_SCALE      # [B, H, keys, D]
        else:
            x = x.float().flatten(1, 2).transpose(1, 2)
        kv.append(x)
    i = torch.arange(Q, device=DEV)
    row = (first[:, None] + torch.minimum(i, ql[:, None] - 1)).flatten()
    q = st["q"][row].float().view(B, Q, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).flatten(2, 3)
    s = (q @ kv[0].transpose(-1, -2)).view(B, hkv, hq // hkv, Q, -1) * st["scale"]
    if case["softcap"]:
        s = case["softcap"] * torch.tanh(s / case["softcap"])
    pos = (lens - ql)[:, None] + i
    key = torch.arange(s.shape[-1], device=DEV)
    far = key - pos[..., None]                                                     # [B, Q, keys]
    if case["alibi"]:
        s = s + st["slopes"].view(hkv, -1, 1, 1) * far[:, None, None].float()
    dead = far > 0
    if case["window"]:
        dead = dead | (far <= -case["window"])
    s = s.masked_fill(dead[:, None, None], -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    del s
    p = p / p.sum(-1, keepdim=True)
    # blocks past a short sequence's end belong to others: their weight is zero
    o = (p.flatten(2, 3) @ kv[1]).view(B, hkv, hq // hkv, Q, d).permute(0, 3, 1, 2, 4).reshape(B, Q, hq, d)
    live = i < ql[:, None]
    dst[row[live.flatten()]] = o[live].to(dst.dtype)


def _plain_attn(st):
    out = torch.empty_like(st["q"])
    c = st["case"]["chunks"]
    _plain_group(st, 0, c, out)
    _plain_group(st, c, len(st["rows"]), out)
    return out


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------
def _own_append(st):
    import paged_kv_attention_decode_gb300 as pa

    case, (kc, vc) = st["case"], st["pools"]
    if case["cache"] == "same":
        q = pa.paged_rope_kv_write(st["q"], st["k"], st["v"], kc, vc, st["slots"], st["pos"], st["table"],
                                   interleaved=case["inter"])
        return [q, kc, vc]
    if case["cache"] == "fp8":
        q = pa.paged_rope_kv_write_fp8(st["q"], st["k"], st["v"], kc, vc, st["slots"], st["pos"], st["table"],
                                       KV8_SCALE, KV8_SCALE, interleaved=case["inter"])
        return [q, kc.view(torch.float8_e4m3fn), vc.view(torch.float8_e4m3fn)]
    if case["rot"]:
        q = pa.paged_rope_kv_write_fp4(st["q"], st["k"], st["v"], kc, vc, st["slots"], st["pos"], st["table"],
                                       KV4_SCALE, KV4_SCALE, interleaved=case["inter"])
    else:
        pa.paged_kv_write_fp4(st["k"], st["v"], kc, vc, st["slots"], KV4_SCALE, KV4_SCALE)
    got = list(pa.paged_kv_unpack_fp4(kc, vc, KV4_SCALE, KV4_SCALE, st["q"].dtype))
    return [q, *got] if case["rot"] else got


def _own_attn(st):
    import paged_kv_attention_decode_gb300 as pa

    case, (kc, vc) = st["case"], st["pools"]
    varlen = case["chunks"] > 0 or case["verify"] > 1
    max_q = max(r[1] for r in st["rows"])
    if case["op"] == "fp4":
        if varlen:
            return pa.paged_attention_prefill_fp4(st["q"], kc, vc, st["tables"], st["lens"], st["cu"], st["scale"],
                                                  KV4_SCALE, KV4_SCALE, max_q, st["max_len"],
                                                  chunk_kv_tokens=st["chunk_kv"])
        return pa.paged_attention_decode_fp4(st["q"], kc, vc, st["tables"], st["lens"], st["scale"], KV4_SCALE,
                                             KV4_SCALE, st["max_len"])
    if varlen:
        return pa.paged_attention_prefill_mod(st["q"], kc, vc, st["tables"], st["lens"], st["cu"], st["scale"], max_q,
                                              st["max_len"], softcap=case["softcap"], window=case["window"],
                                              alibi_slopes=st["slopes"])
    return pa.paged_attention_decode_mod(st["q"], kc, vc, st["tables"], st["lens"], st["scale"], st["max_len"],
                                         softcap=case["softcap"], window=case["window"], alibi_slopes=st["slopes"])


def run(state):
    if state["case"]["op"] == "append":
        return _own_append(state) if own else _plain_append(state)
    return _own_attn(state) if own else _plain_attn(state)


# ---------------------------------------------------------------------------
# bytes and operations that a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "append":
        T, nb = case["T"], (case["T"] + BS - 1) // BS + 4
        row = {"same": 2 * d, "fp8": d, "fp4": d // 2 + d // 16}[case["cache"]]
        b = T * (2 * hkv * (2 * d + row) + 8)
        if case["rot"]:
            b += T * (4 * hq * d + 4 * case["rot"] + 8)
        if case["cache"] == "fp4":       # the pools read back as values
            b += nb * BS * 2 * hkv * (row + 2 * d)
        return {"bytes": b, "flops": 3 * T * case["rot"] * (hq + hkv) + 4 * T * hkv * d}
    b, f = 0, 0
    for n, c in _lens(case):
        w = case["window"] or n + 1
        lo = max(0, n - c + 1 - w)                                            # first key that any row sees
        b += (n - lo) * 2 * hkv * (d // 2 + d // 16 if case["op"] == "fp4" else 2 * d) + 4 * c * hq * d
        seen = sum(min(n - c + 1 + i, w) for i in range(c))
        f += 4 * hq * d * seen
    return {"bytes": b, "flops": f}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _nearest(x, grid):
    """Nearest value of an ascending grid to each |x|, ties to the even index, past its end the last; signed."""
    g = torch.tensor(grid, dtype=torch.float64, device=x.device)
    a = x.abs().clamp(max=float(g[-1]))
    hi = torch.searchsorted(g, a).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = g[hi] - a, a - g[lo]
    take_hi = (up < down) | ((up == down) & (hi % 2 == 0))
    return torch.where(take_hi, g[hi], g[lo]) * torch.sign(x)


def _e4m3_grid():
    return [m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1]


def _exact_rotate(x, pos, table, rot, inter):
    half = rot // 2
    y = x.clone()
    c, s = table[pos, :half].double().unsqueeze(1), table[pos, half:].double().unsqueeze(1)
    i = torch.arange(half, device=x.device)
    ia, ib = (2 * i, 2 * i + 1) if inter else (i, i + half)
    y[:, :, ia] = x[:, :, ia] * c - x[:, :, ib] * s
    y[:, :, ib] = x[:, :, ia] * s + x[:, :, ib] * c
    return y


def _exact_decode4(tiles, d, v):
    """Values of tiles [n, H, bytes] as [n, H, 16, D], in 64 bits."""
    n, h, _ = tiles.shape
    out = torch.empty(n, h, BS, d, dtype=torch.float64, device=tiles.device)
    g2 = torch.tensor(E2M1, dtype=torch.float64, device=tiles.device)
    g8 = torch.tensor(_e4m3_grid() + [math.nan], dtype=torch.float64, device=tiles.device)
    code = tiles[:, :, :BS * d // 2].reshape(n, h, BS, d // 2).long()
    sc = g8[tiles[:, :, BS * d // 2:].long()]
    sc = sc.reshape(n, h, d // 16, BS).permute(0, 1, 3, 2) if v else sc.reshape(n, h, BS, d // 16)
    for part in (0, 1):
        c = (code >> (4 * part)) & 15
        val = g2[c & 7] * (1 - 2 * (c >> 3))
        out[..., part::2] = val * sc.repeat_interleave(8, -1)
    return out


def _exact_append(case, st):
    q, k, v = st["q"].double(), st["k"].double(), st["v"].double()
    d, hkv = case["d"], case["hkv"]
    if case["rot"]:
        q = _exact_rotate(q, st["pos"], st["table"], case["rot"], case["inter"])
        k = _exact_rotate(k, st["pos"], st["table"], case["rot"], case["inter"])
    live = torch.nonzero(st["slots"] >= 0).flatten()
    slot = st["slots"][live]
    got = []
    for x, pool, isv in ((k, st["pools"][0], False), (v, st["pools"][1], True)):
        if case["cache"] == "fp8":
            x = _nearest(x / KV8_SCALE, _e4m3_grid())
            base = pool.view(torch.float8_e4m3fn).double().transpose(1, 2)
        elif case["cache"] == "fp4":
            y = (x / KV4_SCALE).reshape(-1, hkv, d // 16, 16)
            s = _nearest(y.abs().amax(-1) / 6.0, _e4m3_grid()).unsqueeze(-1)
            y = torch.where(s > 0, _nearest(y / s.clamp(min=1e-30), E2M1) * s, torch.zeros_like(y))
            x = y.reshape(-1, hkv, d) * KV4_SCALE
            base = _exact_decode4(pool, d, isv).transpose(1, 2) * KV4_SCALE
        else:
            base = pool.double()
        flat = base.reshape(-1, hkv, d).clone()
        flat[slot] = x[live]
        flat = flat.reshape(-1, BS, hkv, d)
        got.append(flat.transpose(1, 2).contiguous() if case["cache"] == "fp8" else flat)
    return [q, *got] if case["rot"] else got


def _exact_attn(case, st):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    q = st["q"].double()
    out = torch.empty_like(q)
    at = 0
    for b, (n, c) in enumerate(st["rows"]):
        ids = st["tables"][b, :(n + BS - 1) // BS].long()
        qs = q[at:at + c].transpose(0, 1)                                      # [Hq, c, D]
        pos = torch.arange(n - c, n, device=DEV)[:, None]
        j = torch.arange(n, device=DEV)[None]
        for h in range(hkv):
            if case["op"] == "fp4":
                kk, vv = (_exact_decode4(p[ids, h:h + 1], d, isv)[:, 0].reshape(-1, d)[:n] * KV4_SCALE
                          for p, isv in zip(st["pools"], (False, True)))
            else:
                kk, vv = (p[ids, :, h].double().reshape(-1, d)[:n] for p in st["pools"])
            hs = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            s = torch.matmul(qs[hs], kk.T) * st["scale"]
            if case["softcap"]:
                s = case["softcap"] * torch.tanh(s / case["softcap"])
            if case["alibi"]:
                s = s - st["slopes"][hs].double()[:, None, None] * (pos - j)
            see = j <= pos
            if case["window"]:
                see = see & (pos - j < case["window"])
            w = torch.softmax(torch.where(see, s, -math.inf), -1)
            out[at:at + c, hs] = torch.matmul(w, vv).transpose(0, 1)
        at += c
    return out


def exact(case, seed):
    st = prepare(case, seed)
    return _exact_append(case, st) if case["op"] == "append" else _exact_attn(case, st)
