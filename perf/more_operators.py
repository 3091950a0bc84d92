"""Cases of beam search over a paged cache and of cross attention.

Each case is one call that a sequence-to-sequence server makes in a step:
cross attention of decoder rows to an encoder's cached states, the selection
of the best continuations over beams and vocabulary, and the reordering of the
block tables and caches that follows it.  `run` computes a case in plain torch
operations, or, with `own` true, through this package's entry points; `exact`
gives the same outputs from the definitions in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False
DEV = "cuda"
BS = 16
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _named(name, c):
    return dict(c, name=name) if name else c


def _cross(name, seqs, lo, hi, hq, hkv, d, dt, plan_seed, rows=0, chunks=0, chunk=0):
    """`rows` queries for each sequence; or, with `chunks`, that many sequences of
    9 to `chunk` queries and 1 to 8 for each of the others."""
    return _named(name, {"op": "cross", "seqs": seqs, "lo": lo, "hi": hi, "hq": hq, "hkv": hkv, "d": d, "dt": dt,
                         "plan_seed": plan_seed, "rows": rows, "chunks": chunks, "chunk": chunk})


def _select(name, seqs, beams, vocab, k, dt, ended=False, masked=0.0):
    return _named(name, {"op": "select", "seqs": seqs, "beams": beams, "vocab": vocab, "k": k, "dt": dt,
                         "ended": ended, "masked": masked})


def _reorder(name, seqs, beams, lo, hi, own_blocks, layers, hkv, d, dt, plan_seed):
    return _named(name, {"op": "reorder", "seqs": seqs, "beams": beams, "lo": lo, "hi": hi,
                         "own_blocks": own_blocks, "layers": layers, "hkv": hkv, "d": d, "dt": dt,
                         "plan_seed": plan_seed})


def listed():
    return [
        # one request's four beams on 1200 states, heads of 64: the latency of a step
        _cross("cross_1x4_beams", 1, 1200, 1200, 12, 12, 64, "f16", 1, rows=4),
        # 64 requests of four beams, grouped heads
        _cross("cross_64x4_beams", 64, 512, 4096, 32, 8, 128, "bf16", 2, rows=4),
        # 128 greedy rows, a KV head for each query head
        _cross("cross_128x1_rows", 128, 128, 2048, 32, 32, 128, "f16", 3, rows=1),
        # the decoder's prompts, and the training-like case of whole targets: long and odd chunks
        _cross("cross_16_chunks", 16, 100, 4096, 32, 8, 128, "bf16", 4, chunks=16, chunk=1024),
        # a continuous-batching step: a few prompts beside beams; some encoders with very few states, some with none
        _cross("cross_step_mixed", 48, 0, 1500, 16, 16, 64, "f16", 5, chunks=4, chunk=300),
        # one request's first candidates: latency
        _select("select_1x4_32000", 1, 4, 32000, 8, "f16"),
        # an odd vocabulary in 32 bits, some beams ended, two thirds of the tokens not allowed
        _select("select_16x5_50001", 16, 5, 50001, 5, "f32", ended=True, masked=0.66),
        # 64 requests of eight beams over a large vocabulary
        _select("select_64x8_131072", 64, 8, 131072, 16, "bf16"),
        # one request of four beams, a small decoder of six layers
        _reorder("reorder_1x4_6_layers", 1, 4, 100, 400, 4, 6, 8, 64, "f16", 6),
        # 64 requests of eight beams, four layers of sixteen heads
        _reorder("reorder_64x8_4_layers", 64, 8, 600, 1100, 4, 4, 16, 128, "bf16", 7),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["cross", "cross", "cross", "select", "select", "reorder"])
    seed = rng.randrange(1 << 20)
    if op == "select":
        seqs, beams = _log(rng, 1, 64), rng.randint(1, 12)
        dt = rng.choice(["f16", "bf16", "f32"])
        vocab = _log(rng, 1000, min(262144, 64 * 8 * 131072 // (seqs * beams * (2 if dt == "f32" else 1))))
        return _select(None, seqs, beams, vocab, rng.choice([1, 2, beams, 2 * beams]), dt,
                       beams > 1 and rng.random() < 0.3, rng.choice([0.0, 0.0, 0.9]))
    hq, hkv = rng.choice([(32, 32), (32, 8), (64, 8), (8, 8), (12, 4), (16, 2), (6, 2), (12, 12)])
    d, dt = rng.choice([64, 128]), rng.choice(["f16", "bf16"])
    if op == "reorder":
        seqs, beams = _log(rng, 1, 64), rng.randint(2, 8)
        lo = _log(rng, 33, 1000)
        layers = rng.randint(1, max(1, min(12, 64 * 8 * 4 * 16 // (seqs * beams * hkv))))
        return _reorder(None, seqs, beams, lo, lo + _log(rng, 1, 1000), rng.randint(1, 4), layers, hkv, d, dt, seed)
    seqs = _log(rng, 1, 128)
    hi = _log(rng, 20, min(8192, max(64, 128 * 2048 * 32 // (seqs * hkv))))
    lo = rng.choice([0, 1, hi // 8, hi])
    if rng.random() < 0.6:
        return _cross(None, seqs, lo, hi, hq, hkv, d, dt, seed, rows=rng.randint(1, 8))
    seqs = min(seqs, 64)
    chunks = rng.randint(1, min(seqs, 16))
    return _cross(None, seqs, lo, min(hi, 4096), hq, hkv, d, dt, seed, chunks=chunks, chunk=_log(rng, 9, 1024))


def _rows(case):
    """(encoder states, queries) of every sequence of a cross attention case: chunks first."""
    rng = random.Random(case["plan_seed"])
    n = [rng.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])]
    if not case["chunks"]:
        return [(x, case["rows"]) for x in n]
    return [(x, _log(rng, 9, case["chunk"]) if i < case["chunks"] else rng.randint(1, 8)) for i, x in enumerate(n)]


def _beams(case):
    """(length, parents) of every request of a reordering case."""
    rng = random.Random(case["plan_seed"])
    return [(rng.randint(case["lo"], case["hi"]), [rng.randrange(case["beams"]) for _ in range(case["beams"])])
            for _ in range(case["seqs"])]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(g, *shape, dt=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).to(dt)


def _pool(g, nb, hkv, d, dt):
    pool = torch.empty(nb, BS, hkv, d, dtype=dt, device=DEV)
    step = max(1, (1 << 27) // (BS * hkv * d))
    for b in range(0, nb, step):
        pool[b:b + step] = _randn(g, min(step, nb - b), BS, hkv, d)
    return pool


def _prepare_cross(case, seed):
    g = _gen(seed)
    rows = _rows(case)
    hq, hkv, d, dt = case["hq"], case["hkv"], case["d"], TYPES[case["dt"]]
    used = [(n + BS - 1) // BS for n, _ in rows]
    nb = int(sum(used) * 1.1) + 4
    perm = torch.randperm(nb, generator=g, device=DEV).to(torch.int32)
    tables = torch.zeros(len(rows), max(1, max(used)), dtype=torch.int32, device=DEV)
    at = 0
    for b, u in enumerate(used):
        tables[b, :u] = perm[at:at + u]
        at += u
    cu = [0]
    for _, c in rows:
        cu.append(cu[-1] + c)
    return {"q": _randn(g, cu[-1], hq, d, dt=dt), "k": _pool(g, nb, hkv, d, dt), "v": _pool(g, nb, hkv, d, dt),
            "tables": tables, "lens": torch.tensor([n for n, _ in rows], dtype=torch.int32, device=DEV), "rows": rows,
            "cu": torch.tensor(cu, dtype=torch.int32, device=DEV) if case["chunks"] else None,
            "scale": 1.0 / math.sqrt(d), "max_len": max(n for n, _ in rows), "max_q": max(c for _, c in rows)}


def _prepare_select(case, seed):
    g = _gen(seed)
    S, W, V = case["seqs"], case["beams"], case["vocab"]
    x = _randn(g, S * W, V) * 3
    # a few tokens that the model favours, the same ones for the beams of a request more often than not
    liked = torch.randint(0, V, (S * W, 20), generator=g, device=DEV)
    liked[:, :10] = liked[::W, :10].repeat_interleave(W, 0)
    x.scatter_add_(1, liked, 8 + 2 * _randn(g, S * W, 20))
    if case["masked"]:
        dead = torch.rand(S * W, V, generator=g, device=DEV) < case["masked"]
        dead[:, :64] = False
        x = x.masked_fill(dead, -math.inf)
    scores = -10 + 2 * _randn(g, S, W)
    ended = None
    if case["ended"]:
        ended = (torch.rand(S, W, generator=g, device=DEV) < 0.3).to(torch.uint8)
        ended[:, 0] = 0                # a live beam is left in every request
    return {"logits": x.to(TYPES[case["dt"]]), "scores": scores, "ended": ended, "end": 2}


def _prepare_reorder(case, seed):
    g = _gen(seed)
    plan = _beams(case)
    W, hkv, d, dt = case["beams"], case["hkv"], case["d"], TYPES[case["dt"]]
    own_blocks = case["own_blocks"]
    # the prompt's blocks are the request's, its last ones each beam's own, with two more for what comes
    full = [n // BS for n, _ in plan]
    shared = [max(0, f + 1 - own_blocks) for f in full]
    nb = sum(s + W * (f + 3 - s) for f, s in zip(full, shared))
    perm = torch.randperm(nb, generator=g, device=DEV).to(torch.int32)
    tables = torch.zeros(len(plan), W, max(full) + 3, dtype=torch.int32, device=DEV)
    at = 0
    for r, (f, s) in enumerate(zip(full, shared)):
        tables[r, :, :s] = perm[at:at + s]
        at += s
        n = f + 3 - s
        tables[r, :, s:s + n] = perm[at:at + W * n].view(W, n)
        at += W * n
    tables = tables.flatten(0, 1).contiguous()
    return {"tables": tables, "out": torch.empty_like(tables),
            "lens": torch.tensor([n for n, _ in plan for _ in range(W)], dtype=torch.int32, device=DEV),
            "parents": torch.tensor([p for _, p in plan], dtype=torch.int32, device=DEV),
            "k": [_pool(g, nb, hkv, d, dt) for _ in range(case["layers"])],
            "v": [_pool(g, nb, hkv, d, dt) for _ in range(case["layers"])]}


def prepare(case, seed):
    st = {"cross": _prepare_cross, "select": _prepare_select, "reorder": _prepare_reorder}[case["op"]](case, seed)
    st["case"] = case
    return st


# ---------------------------------------------------------------------------
# plain forms: 32 bits (64 where scores are compared), rounded once at the end
# ---------------------------------------------------------------------------
def _plain_group(st, b0, b1, dst):
    """Cross attention of sequences b0..b1-1, padded to their most states and queries."""
    case, rows = st["case"], st["rows"][b0:b1]
    if not rows:
        return
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    first = sum(c for _, c in st["rows"][:b0])
    B, N, Q = len(rows), max(1, max(n for n, _ in rows)), max(c for _, c in rows)
    tab = st["tables"][b0:b1, :(N + BS - 1) // BS].long()
    lens = st["lens"][b0:b1].long()
    ql = torch.tensor([c for _, c in rows], device=DEV)
    i = torch.arange(Q, device=DEV)
    row = (first + (ql.cumsum(0) - ql)[:, None] + torch.minimum(i, ql[:, None] - 1)).flatten()
    k, v = (p[tab].float().flatten(1, 2).transpose(1, 2) for p in (st["k"], st["v"]))     # [B, H, states, D]
    q = st["q"][row].float().view(B, Q, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).flatten(2, 3)
    s = (q @ k.transpose(-1, -2)) * st["scale"]                                           # [B, H, G Q, states]
    dead = torch.arange(s.shape[-1], device=DEV) >= lens[:, None]
    s = s.masked_fill(dead[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    del s
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-30)       # no states: a row of zeros
    o = (p @ v).view(B, hkv, hq // hkv, Q, d).permute(0, 3, 1, 2, 4).reshape(B, Q, hq, d)
    live = i < ql[:, None]
    dst[row[live.flatten()]] = o[live].to(dst.dtype)


def _plain_cross(st):
    out = torch.empty_like(st["q"])
    c = st["case"]["chunks"]
    for b in range(c):                       # long chunks one by one, the others together
        _plain_group(st, b, b + 1, out)
    _plain_group(st, c, len(st["rows"]), out)
    return out


def _plain_select(st):
    case, ended = st["case"], st["ended"]
    S, W, V, k = case["seqs"], case["beams"], case["vocab"], case["k"]
    x = st["logits"].double()
    x = x - x.amax(-1, keepdim=True)
    x -= torch.log(torch.exp(x).sum(-1, keepdim=True))
    x += st["scores"].double().view(S * W, 1)
    if ended is not None:
        e = ended.view(S * W, 1).bool()
        only = torch.arange(V, device=DEV) == st["end"]
        x = torch.where(e, torch.where(only, st["scores"].double().view(S * W, 1), -math.inf), x)
    best, at = torch.sort(x.view(S, W * V), dim=-1, descending=True, stable=True)
    best, at = best[:, :k].float(), at[:, :k]
    parent, token = (at // V).int(), (at % V).int()
    if ended is None:
        return [best, parent, token]
    return [best, parent, token, (ended.gather(1, parent.long()).bool() | (token == st["end"])).to(torch.uint8)]


def _plain_reorder(st):
    case = st["case"]
    S, W = case["seqs"], case["beams"]
    old = st["tables"].view(S, W, -1)
    par = st["parents"].long()
    n = st["lens"].view(S, W)[:, 0].long()
    f, t = n // BS, n % BS
    col = torch.arange(old.shape[2], device=DEV)
    new = torch.where(col < f[:, None, None], old.gather(1, par[..., None].expand_as(old)), old)
    tail = old.gather(2, f[:, None, None].expand(S, W, 1))[..., 0]                 # block f of every row
    beam = torch.arange(W, device=DEV)
    same = par[:, :, None] == par[:, None, :]
    keeps = ~(same & (beam[None, :] < beam[:, None])).any(-1)                      # lowest child of its parent
    childless = ~(par[:, :, None] == beam).any(1)                                  # [S, W]
    free = torch.sort(torch.where(childless, beam, W), -1).values                  # their numbers first
    rank = (~keeps).long().cumsum(1) - 1                                           # of the children that move
    take = torch.where(keeps, par, free.gather(1, rank.clamp(min=0)).clamp(max=W - 1))
    block = torch.where((t > 0)[:, None], tail.gather(1, take), tail)
    new.scatter_(2, f[:, None, None].expand(S, W, 1), block[..., None])
    move = ~keeps & (t > 0)[:, None]
    src, dst = tail.gather(1, par)[move].long(), block[move].long()
    rows = torch.arange(BS, device=DEV) < t[:, None, None].expand(S, W, 1)[move]   # [pairs, 16]
    for pool in st["k"] + st["v"]:
        pool[dst] = torch.where(rows[..., None, None], pool[src], pool[dst])
    return [new.view_as(st["tables"]), *st["k"], *st["v"]]


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------
def _own_cross(st):
    import paged_kv_attention_decode_gb300 as pa

    return pa.paged_cross_attention(st["q"], st["k"], st["v"], st["tables"], st["lens"], st["scale"],
                                    max_enc_len=st["max_len"], cu_q_lens=st["cu"], max_q_len=st["max_q"])


def _own_select(st):
    import paged_kv_attention_decode_gb300 as pa

    return list(pa.beam_select(st["logits"], st["scores"], st["case"]["k"], finished=st["ended"],
                               end_token=st["end"]))


def _own_reorder(st):
    import paged_kv_attention_decode_gb300 as pa

    pa.beam_reorder(st["tables"], st["lens"], st["parents"], st["k"], st["v"], out=st["out"])
    return [st["out"], *st["k"], *st["v"]]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"cross": _own_cross, "select": _own_select, "reorder": _own_reorder}[op](state)
    return {"cross": _plain_cross, "select": _plain_select, "reorder": _plain_reorder}[op](state)


# ---------------------------------------------------------------------------
# bytes and operations that a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    if case["op"] == "select":
        n = case["seqs"] * case["beams"] * case["vocab"]
        return {"bytes": n * (4 if case["dt"] == "f32" else 2) + case["seqs"] * (4 * case["beams"] + 12 * case["k"]),
                "flops": 4 * n}
    if case["op"] == "reorder":
        b = 0
        for n, par in _beams(case):
            copies = case["beams"] - len(set(par)) if n % BS else 0
            b += copies * (n % BS) * case["hkv"] * case["d"] * 2 * 2 * 2 * case["layers"]     # K and V, read and written
            b += case["beams"] * ((n // BS + 3) * 8 + 8)
        return {"bytes": b, "flops": 0}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    b = f = 0
    for n, c in _rows(case):
        b += n * 2 * hkv * d * 2 + 4 * c * hq * d
        f += 4 * hq * d * c * n
    return {"bytes": b, "flops": f}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_cross(case, st):
    hkv, G = case["hkv"], case["hq"] // case["hkv"]
    q = st["q"].double()
    out = torch.zeros_like(q)
    at = 0
    for b, (n, c) in enumerate(st["rows"]):
        ids = st["tables"][b, :(n + BS - 1) // BS].long()
        for h in range(hkv if n else 0):
            kk, vv = (p[ids, :, h].double().reshape(-1, case["d"])[:n] for p in (st["k"], st["v"]))
            w = torch.softmax(torch.einsum("qhd,nd->qhn", q[at:at + c, h * G:(h + 1) * G], kk) * st["scale"], -1)
            out[at:at + c, h * G:(h + 1) * G] = torch.einsum("qhn,nd->qhd", w, vv)
        at += c
    return out


def _exact_select(case, st):
    S, W, V, k = case["seqs"], case["beams"], case["vocab"], case["k"]
    x, cum = st["logits"].view(S, W, V), st["scores"].double()
    best, parent, token, done = np.empty((S, k)), np.empty((S, k), np.int32), np.empty((S, k), np.int32), None
    ended = np.zeros((S, W), bool) if st["ended"] is None else st["ended"].cpu().numpy().astype(bool)
    for s in range(S):
        lp = torch.log_softmax(x[s].double(), -1) + cum[s][:, None]
        for w in range(W):
            if ended[s, w]:
                lp[w] = -math.inf
                lp[w, st["end"]] = cum[s, w]
        lp = lp.flatten()
        border = torch.topk(lp, min(k, lp.numel())).values[-1]
        at = torch.nonzero(lp >= border).flatten().cpu().numpy()
        val = lp[lp >= border].cpu().numpy()
        order = np.lexsort((at, -val))[:k]
        best[s], parent[s], token[s] = val[order], at[order] // V, at[order] % V
    got = [torch.from_numpy(a).to(DEV) for a in (best, parent, token)]
    if st["ended"] is not None:
        done = np.take_along_axis(ended, parent.astype(np.int64), 1) | (token == st["end"])
        got.append(torch.from_numpy(done.astype(np.uint8)).to(DEV))
    return got


def _exact_reorder(case, st):
    W = case["beams"]
    tables = st["tables"].cpu().numpy()
    new = tables.copy()
    copies = []
    for s, (n, parents) in enumerate(_beams(case)):
        f, t = divmod(n, BS)
        taken, spare = set(), [tables[s * W + p, f] for p in range(W) if p not in parents]
        for j, p in enumerate(parents):
            new[s * W + j, :f] = tables[s * W + p, :f]
            if t == 0:
                continue
            if p not in taken:
                taken.add(p)
                new[s * W + j, f] = tables[s * W + p, f]
            else:
                new[s * W + j, f] = spare.pop(0)
                copies.append((int(tables[s * W + p, f]), int(new[s * W + j, f]), t))
    got = [torch.from_numpy(new).to(DEV)]
    for pool in st["k"] + st["v"]:
        p = pool.double()
        for src, dst, t in copies:
            p[dst, :t] = p[src, :t]
        got.append(p)
    return got


def exact(case, seed):
    st = prepare(case, seed)
    return {"cross": _exact_cross, "select": _exact_select, "reorder": _exact_reorder}[case["op"]](case, st)
