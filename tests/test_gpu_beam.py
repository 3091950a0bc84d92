"""Beam selection and reordering against 64-bit references, and a whole beam
search (self attention, cross attention, selection, reordering) over caches."""
import math

import numpy as np
import pytest
import torch

import paged_kv_attention_decode_gb300 as pa
from tests import _beam_ref as B
from tests import _ref64 as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
BLOCK_ID, BEAM = 1, 64
# a score is rounded once (2^-24 of it, counted double for subnormal neighbours
# and the rounded sum's own share); its log-sum-exp is a sum of fp32 exponentials:
# each term within 2^-22 (2^x) and |d| log2(e) 2^-23 ln 2 (the rounded difference
# and product, d < 32 where a term counts), the sum's roundings 48 x 2^-24 (32
# terms a thread, then 13 pairwise steps): together below 160 x 2^-24
LSE_TOL = 160 * 2.0 ** -24


def run(logits, scores, k, finished=None, end_token=-1, **kw):
    got = pa.beam_select(logits, torch.from_numpy(scores).to(DEV), k,
                         finished=None if finished is None else torch.from_numpy(finished).to(DEV),
                         end_token=end_token, **kw)
    torch.cuda.synchronize()
    return got


def check(got, logits, scores, k, finished=None, end_token=-1):
    """logits [S, W, V] in 64 bits, on the CPU."""
    S, W, V = logits.shape
    top = {torch.float16: 65504.0, torch.bfloat16: float(torch.finfo(torch.bfloat16).max),
           torch.float32: float(np.finfo(np.float32).max)}[check.dtype]
    x = logits.double().numpy()
    cand = B.candidate_scores(x, scores, finished, end_token, top).reshape(S, W * V)
    ref, parents, tokens, done = B.select(x, scores, k, finished, end_token, top)
    sc, pr, tk = (t.cpu().numpy() for t in got[:3])
    assert sc.shape == pr.shape == tk.shape == (S, k)
    assert ((pr >= 0) & (pr < W) & (tk >= 0) & (tk < V)).all()
    flat = pr.astype(np.int64) * V + tk
    for s in range(S):
        assert len(set(flat[s])) == k
        mine = cand[s, flat[s]]                                   # exact scores of what was chosen
        with np.errstate(invalid="ignore"):
            tol = LSE_TOL + 2.0 ** -23 * np.abs(mine)
            near = (sc[s] == mine) | (np.abs(sc[s] - mine) <= tol)
        assert near.all(), (sc[s], mine)
        # the k best, in order, wherever the exact scores are apart or exactly equal
        nxt = np.concatenate([ref[s], [np.sort(cand[s])[::-1][k] if k < W * V else -np.inf]])
        for r in range(k):
            if flat[s, r] != parents[s, r] * V + tokens[s, r]:
                gap = abs(mine[r] - ref[s, r])
                assert 0 < gap <= 2 * LSE_TOL, (s, r, mine[r], ref[s, r])
        assert not np.isnan(nxt[:k]).any()
    if finished is not None:
        fin = finished.astype(bool)
        assert np.array_equal(got[3].cpu().numpy().astype(bool), np.take_along_axis(fin, pr, 1) | (tk == end_token))
    else:
        assert len(got) == 3


def make(S, W, V, dt, seed, kind="normal"):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((S, W, V)).astype(np.float32) * 3
    if kind == "peaked":
        x[rng.random((S, W, V)) < 5 / V] += 12
    if kind == "masked":
        x[rng.random((S, W, V)) < 0.98] = -np.inf
    if kind == "equal":
        x[:] = 0.25
    if kind == "steps":                                          # many ties
        x = np.round(x)
    if kind == "sorted":                                         # the best lie side by side
        x = -np.sort(-x, -1)
    check.dtype = dt
    return torch.from_numpy(x).to(dt), (rng.standard_normal((S, W)) * 4 - 10).astype(np.float32)


@pytest.mark.parametrize("kind", ["normal", "peaked", "masked", "equal", "steps", "sorted"])
@pytest.mark.parametrize("dn", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("S,W,V,k", [(1, 1, 1, 1), (1, 4, 7, 8), (3, 5, 1001, 10), (2, 4, 32000, 8), (1, 2, 8193, 64),
                                     (5, 1, 4097, 1), (1, 32, 129, 64), (2, 3, 50001, 6),
                                     (9, 4, 5001, 8), (40, 2, 3001, 4), (2, 12, 150000, 24),
                                     (140, 1, 700, 3), (3, 4, 1000, 24), (2, 1, 1000, 64), (70, 3, 20000, 6)])
def test_select(S, W, V, k, dn, kind):
    x, scores = make(S, W, V, DT[dn], seed=V + k, kind=kind)
    got = run(x.view(S * W, V).to(DEV), scores, k)
    check(got, x, scores, k)


@pytest.mark.parametrize("dn", ["f16", "f32"])
@pytest.mark.parametrize("pad,off", [(0, 1), (5, 3), (8, 8), (1, 0)])
def test_rows_on_any_boundary(dn, pad, off):
    """Strided rows that start anywhere; what lies between them is not read as a logit."""
    S, W, V = 2, 3, 20003
    x, scores = make(S, W, V, DT[dn], seed=pad + off)
    buf = torch.full((S * W * (V + pad) + off + 16,), float("inf"), dtype=DT[dn], device=DEV)
    rows = buf[off:off + S * W * (V + pad)].view(S * W, V + pad)[:, :V]
    rows.copy_(x.view(S * W, V))
    check(run(rows, scores, 6), x, scores, 6)
    check(run(rows.unflatten(0, (S, W)), scores, 6), x, scores, 6)


@pytest.mark.parametrize("dn", ["f16", "bf16", "f32"])
def test_what_is_not_finite(dn):
    S, W, V, k = 4, 3, 5000, 12
    x, scores = make(S, W, V, DT[dn], seed=1)
    x[0, 0, 17] = float("nan")
    x[0, 1, :] = float("nan")
    x[1, 2, 4999] = float("inf")
    x[1, 2, 3] = torch.finfo(DT[dn]).max                         # a tie with it, and lower
    x[2] = -float("inf")
    x[2, 1, 77], x[2, 1, 4000] = 1.0, 1.0
    x[3, 0, :100] = -float("inf")
    scores[3, 1], scores[3, 2] = -np.inf, np.nan
    got = run(x.view(S * W, V).to(DEV), scores, k)
    check(got, x, scores, k)
    sc, pr, tk = (t.cpu().numpy() for t in got)
    assert (pr[2, :2] == 1).all() and list(tk[2, :2]) == [77, 4000]
    assert np.isneginf(sc[2, 2:]).all() and list(tk[2, 2:]) == list(range(k - 2)) and (pr[2, 2:] == 0).all()
    assert (pr[3] == 0).all()
    assert list(tk[1, :2]) == [3, 4999] or pr[1, 0] != 2


@pytest.mark.parametrize("dn", ["f16", "bf16", "f32"])
def test_what_is_not_finite_in_few_logits(dn):
    S, W, V, k = 3, 2, 90, 20
    x, scores = make(S, W, V, DT[dn], seed=9)
    x[0, 0, ::3] = float("nan")
    x[0, 1, 5], x[0, 1, 40] = float("inf"), torch.finfo(DT[dn]).max
    x[1, 0, :80] = -float("inf")
    x[1, 1] = float("nan")
    x[2, :, 1:] = -float("inf")
    fin = np.zeros((S, W), np.uint8)
    fin[2, 1] = 1
    check(run(x.view(S * W, V).to(DEV), scores, k), x, scores, k)
    check(run(x.view(S * W, V).to(DEV), scores, k, fin, 89), x, scores, k, fin, 89)


def test_first_step_and_dead_requests():
    S, W, V, k = 3, 4, 3000, 8
    x, scores = make(S, W, V, torch.float16, seed=2)
    scores[0, 1:] = -np.inf
    scores[1] = -np.inf
    scores[2] = [np.inf, 1.0, 2.0, np.float32(np.finfo(np.float32).max)]
    got = run(x.view(S * W, V).to(DEV), scores, k)
    check(got, x, scores, k)
    assert not got[1][0].any()
    assert torch.equal(got[2][1].cpu(), torch.arange(k, dtype=torch.int32)) and not got[1][1].any()


@pytest.mark.parametrize("kind", [np.uint8, bool])
def test_ended_beams(kind):
    S, W, V, k, end = 4, 4, 2000, 4, 7
    x, scores = make(S, W, V, torch.bfloat16, seed=3)
    fin = np.zeros((S, W), kind)
    fin[0, 2] = fin[1, 0] = fin[1, 3] = 1
    fin[2] = 1
    scores[0, 2] = 3.0                                            # the best there is
    scores[2, 1] = -np.inf                                        # ended and dead
    x[0, 2] = float("nan")                                        # its logits do not count
    x[3, 1, end] = 40                                             # ends now
    got = run(x.view(S * W, V).to(DEV), scores, k, fin, end)
    check(got, x, scores, k, fin, end)
    assert (int(got[1][0, 0]), int(got[2][0, 0]), float(got[0][0, 0])) == (2, end, 3.0)
    assert got[3].dtype == (torch.uint8 if kind is np.uint8 else torch.bool)
    assert bool(got[3][2].any()) and float(got[0][2, 3]) == -math.inf


@pytest.mark.parametrize("V", [40, 5000])
@pytest.mark.parametrize("dn", ["bf16", "f32"])
def test_scores_and_logits_at_the_ends_of_the_range(dn, V):
    """Sums past fp32's range on the way, and scores below it; ended beams beside them."""
    S, W, k = 5, 3, 9
    x, scores = make(S, W, V, DT[dn], seed=V)
    big, top = 2.0 ** 127, float(np.finfo(np.float32).max)
    x[0, 0, 7], x[0, 1, 11] = big, -big                           # one huge logit: the others are far below it
    scores[0] = [-big, 1.0, -1.5 * big]
    x[1] = x[1] * 2.0 ** 120
    scores[1] = [top, -top, 0.0]
    scores[2] = [-top, -top, -top]
    x[3, 1] = -big                                                # equal ones
    scores[3] = [-5.0, big, 2.0]
    x[4, 0, ::2] = -big
    scores[4] = [0.0, -big, top]
    fin = np.zeros((S, W), np.uint8)
    fin[0, 2] = fin[1, 1] = fin[3, 2] = fin[4, 2] = 1
    check(run(x.view(S * W, V).to(DEV), scores, k), x, scores, k)
    check(run(x.view(S * W, V).to(DEV), scores, k, fin, 3), x, scores, k, fin, 3)


@pytest.mark.parametrize("dn", ["f16", "f32"])
@pytest.mark.parametrize("logit", [0.0, 3.5, -7.0])
@pytest.mark.parametrize("V", [1, 3, 700, 70_000])
def test_one_token_allowed(V, logit, dn):
    """A forced token costs nothing: the beam's score comes back as it was, 0 as 0."""
    S, W = 4, 5
    x = torch.full((S, W, V), -float("inf"), dtype=DT[dn])
    tok = np.random.default_rng(V).integers(0, V, (S, W))
    for s in range(S):
        for w in range(W):
            x[s, w, tok[s, w]] = logit
    scores = np.zeros((S, W), np.float32)
    scores[1] = [-1, -2, 0, -3, -4]
    scores[2, 1:] = -np.inf
    scores[3] = -np.float32(1e-40)
    check.dtype = DT[dn]
    for k in (1, 2, 5):
        got = run(x.view(S * W, V).to(DEV), scores, min(k, W * V))
        check(got, x, scores, min(k, W * V))
        assert float(got[0][0, 0]) == 0 and int(got[1][0, 0]) == 0 and int(got[2][0, 0]) == tok[0, 0]
        assert float(got[0][1, 0]) == 0 and int(got[1][1, 0]) == 2
        assert float(got[0][2, 0]) == 0 and int(got[2][2, 0]) == tok[2, 0]


def test_equal_rows_prefer_the_lower_beam():
    S, W, V, k = 2, 6, 999, 12
    x, scores = make(S, 1, V, torch.float32, seed=4)
    x = x.expand(S, W, V).contiguous()
    scores = np.repeat(scores, W, 1)
    got = run(x.view(S * W, V).to(DEV), scores, k)
    check(got, x, scores, k)
    assert got[1].cpu().tolist() == [[0, 1, 2, 3, 4, 5] * 2] * S


def test_largest_vocabulary_and_many_requests():
    x, scores = make(1, 2, 1 << 20, torch.float32, seed=5)
    buf = torch.empty(2 * (1 << 20) + 3, device=DEV)[3:].view(2, 1 << 20)
    check(run(buf.copy_(x[0]), scores, 64), x, scores, 64)
    x, scores = make(700, 3, 65, torch.float16, seed=6)
    check(run(x.view(-1, 65).to(DEV), scores, 6), x, scores, 6)


def test_select_same_results_every_time_and_captured():
    S, W, V, k = 8, 4, 30011, 8
    x, scores = make(S, W, V, torch.float16, seed=7, kind="steps")
    xd, sd = x.view(S * W, V).to(DEV), torch.from_numpy(scores).to(DEV)
    first = pa.beam_select(xd, sd, k)
    ws = torch.empty(pa.beam_select_workspace_bytes(S, W, V, k, torch.float16), dtype=torch.uint8, device=DEV)
    out = tuple(torch.empty_like(t) for t in first)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.beam_select(xd, sd, k, out=out, workspace=ws)
    for i in range(5):
        xd.copy_(xd.flip(0))
        want = pa.beam_select(xd, sd, k, workspace=ws)
        g.replay()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        other = pa.beam_select(xd, sd, k, stream=side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(out, want, other))
    check(want, x.flip(0, 1), scores, k)


def test_select_in_place_and_captured():
    """With as many results as beams, scores and flags take the results' place:
    replays go on from one another."""
    S, W, V, end = 3, 4, 1500, 9
    x, scores = make(S, W, V, torch.float16, seed=8, kind="peaked")
    xd = x.view(S * W, V).to(DEV)
    cum, fin = torch.from_numpy(scores).to(DEV), torch.zeros((S, W), dtype=torch.uint8, device=DEV)
    par, tok = torch.empty((S, W), dtype=torch.int32, device=DEV), torch.empty((S, W), dtype=torch.int32, device=DEV)
    ws = torch.empty(pa.beam_select_workspace_bytes(S, W, V, W, torch.float16), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.beam_select(xd, cum, W, finished=fin, end_token=end, out=(cum, par, tok, fin), workspace=ws)
    for step in range(6):
        before, ended = cum.cpu().numpy().copy(), fin.cpu().numpy().copy()
        if step == 3:                                        # a request without candidates: its flags stay with the fill
            before[1], ended[1] = -np.inf, [1, 0, 1, 0]
            cum[1], fin[1] = torch.from_numpy(before[1]).to(DEV), torch.from_numpy(ended[1]).to(DEV)
        xd.copy_(torch.from_numpy(np.roll(x.view(S * W, V).float().numpy(), step, 1)).half())
        g.replay()
        torch.cuda.synchronize()
        check((cum, par, tok, fin), xd.view(S, W, V).cpu(), before, W, ended, end)


def test_select_ranks_what_fp32_does_not_tell_apart():
    """Two beams whose best differ by less than a unit of the fp32 score."""
    S, W, V = 1, 2, 64
    x = torch.full((S, W, V), -30.0)
    x[0, 0, 5], x[0, 1, 9] = 0.0, 0.0
    check.dtype = torch.float32
    a = np.float32(-1000.0)
    for first in (0, 1):
        scores = np.full((S, W), a)
        x[0, first, 20:] = -12.0                             # more mass elsewhere: a lower score, by 44 e^-12
        x[0, 1 - first, 20:] = -30.0
        sc, par, tok = run(x.view(W, V).to(DEV), scores, 2)
        assert par[0].tolist() == [1 - first, first] and tok[0].tolist() == [9 if first == 0 else 5, 5 if first == 0 else 9]


# ---------------------------------------------------------------------------
# reordering
# ---------------------------------------------------------------------------
def beams(lens, W, spare, seed, parents=None):
    """Tables of S requests of W rows: shared whole blocks up to half the length, then each row its own."""
    rng = np.random.default_rng(seed)
    S, mb = len(lens), max(int(n) // 16 for n in lens) + 1 + spare
    perm = list(rng.permutation(S * (W + 1) * mb + 3))
    tables = np.zeros((S, W, mb), np.int32)
    for s, n in enumerate(lens):
        shared = int(n) // 32
        tables[s, :, :shared] = [perm.pop() for _ in range(shared)]
        for w in range(W):
            tables[s, w, shared:] = [perm.pop() for _ in range(mb - shared)]
    if parents is None:
        parents = rng.integers(0, W, (S, W))
    return tables, np.asarray(parents, np.int32), S * (W + 1) * mb + 3


def pools_of(kind, nb, layers, H, D, seed):
    g = torch.Generator().manual_seed(seed)
    shape = {"f16": (nb, 16, H, D), "bf16": (nb, 16, H, D), "fp8": (nb, H, 16, D), "fp4": (nb, H, 9 * D)}[kind]
    dt = {"f16": torch.float16, "bf16": torch.bfloat16}.get(kind, torch.uint8)
    raw = [[torch.randint(0, 256, (*shape[:-1], shape[-1] * dt.itemsize), dtype=torch.uint8, generator=g).view(dt)
            for _ in range(layers)] for _ in range(2)]
    return raw


def bytes_of(t):
    return t.contiguous().view(torch.uint8).cpu()


def expect(pool, copies, kind):
    p = pool.clone()
    for src, dst, t in copies:
        if kind == "fp4":
            p[dst] = p[src]
        elif kind == "fp8":
            p[dst, :, :t] = p[src, :, :t]
        else:
            p[dst, :t] = p[src, :t]
    return p


def reorder(tables, lens, parents, ks, vs, out=None, **kw):
    S, W, mb = tables.shape
    t = torch.from_numpy(tables).to(DEV).view(S * W, mb)
    n = torch.tensor(np.repeat(lens, W).astype(np.int32), device=DEV)
    got = pa.beam_reorder(t, n, torch.from_numpy(parents).to(DEV), ks, vs, out=t if out is None else out, **kw)
    torch.cuda.synchronize()
    return got.cpu().numpy().reshape(S, W, mb)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("kind,H,D", [("f16", 3, 64), ("bf16", 8, 128), ("fp8", 5, 128), ("fp4", 2, 128),
                                      ("fp4", 3, 64)])
@pytest.mark.parametrize("W", [1, 2, 5, 8, 32])
def test_reorder(W, kind, H, D, in_place):
    lens = [0, 1, 15, 16, 17, 100, 320, 333]
    tables, parents, nb = beams(lens, W, 2, seed=W)
    ks, vs = pools_of(kind, nb, 3, H, D, seed=W)
    kd, vd = [x.to(DEV) for x in ks], [x.to(DEV) for x in vs]
    out = None if in_place else torch.full(tables.shape, -7, dtype=torch.int32, device=DEV).flatten(0, 1)
    got = reorder(tables, lens, parents, kd, vd, out)
    new, copies = B.reorder(tables, lens, parents)
    assert np.array_equal(got, new)
    for a, b in zip(ks + vs, kd + vd):
        assert torch.equal(bytes_of(expect(a, copies, kind)), bytes_of(b))
    assert pa.device_error() == 0


@pytest.mark.parametrize("parents", [[0, 1, 2, 3], [3, 2, 1, 0], [2, 2, 2, 2], [1, 1, 3, 3], [0, 0, 0, 1]])
def test_reorder_families(parents):
    tables, par, nb = beams([70], 4, 1, seed=1, parents=[parents])
    (k,), (v,) = pools_of("f16", nb, 1, 2, 64, seed=1)
    kd, vd = k.to(DEV), v.to(DEV)
    got = reorder(tables, [70], par, kd, vd)
    new, copies = B.reorder(tables, [70], par)
    assert np.array_equal(got, new) and len(set(new[0, :, 4])) == 4
    assert torch.equal(bytes_of(expect(k, copies, "f16")), bytes_of(kd))
    assert torch.equal(bytes_of(expect(v, copies, "f16")), bytes_of(vd))


def test_reorder_many_layers_and_none():
    lens, W = [40, 90], 3
    tables, parents, nb = beams(lens, W, 0, seed=3)
    ks, vs = pools_of("f16", nb, 70, 1, 64, seed=3)
    kd, vd = [x.to(DEV) for x in ks], [x.to(DEV) for x in vs]
    new, copies = B.reorder(tables, lens, parents)
    assert np.array_equal(reorder(tables, lens, parents, kd, vd), new)
    for a, b in zip(ks + vs, kd + vd):
        assert torch.equal(bytes_of(expect(a, copies, "f16")), bytes_of(b))
    assert np.array_equal(reorder(tables, lens, parents, [], []), new)
    out = torch.zeros(tables.shape, dtype=torch.int32, device=DEV).flatten(0, 1)
    assert np.array_equal(reorder(tables, lens, parents, [], [], out), new)
    assert pa.device_error() == 0


@pytest.mark.parametrize("what,flag", [("parent", BEAM), ("negative", BEAM), ("length", BEAM), ("long", BEAM),
                                       ("twin", BEAM), ("block", BLOCK_ID)])
@pytest.mark.parametrize("in_place", [True, False])
def test_requests_that_cannot_be_reordered_stay(what, flag, in_place):
    lens, W = [40, 90, 21], 4
    tables, parents, nb = beams(lens, W, 1, seed=4)
    parents[1] = [0, 0, 1, 1]
    (k,), (v,) = pools_of("bf16", nb, 1, 2, 64, seed=4)
    kd, vd = k.to(DEV), v.to(DEV)
    mb = tables.shape[2]
    n = np.repeat(lens, W).astype(np.int32)
    if what == "parent":
        parents[1, 3] = W
    elif what == "negative":
        parents[1, 0] = -1
    elif what == "length":
        n[W + 2] = 91
    elif what == "long":
        n[W:2 * W] = mb * 16 + 1
    elif what == "twin":
        tables[1, 2, 5] = tables[1, 0, 5]
    else:
        tables[1, 3, 5] = nb
    t = torch.from_numpy(tables).to(DEV).flatten(0, 1)
    out = t if in_place else torch.empty_like(t)
    pa.beam_reorder(t, torch.from_numpy(n).to(DEV), torch.from_numpy(parents).to(DEV), kd, vd, out=out)
    torch.cuda.synchronize()
    assert pa.device_error() == flag
    p2 = parents.copy()
    p2[1] = np.arange(W)                                          # as it was
    new, copies = B.reorder(tables, lens, p2)
    assert np.array_equal(out.cpu().numpy().reshape(tables.shape), new)
    assert torch.equal(bytes_of(expect(k, copies, "bf16")), bytes_of(kd))


def test_reorder_on_a_given_stream():
    lens, W = [37, 200], 4
    tables, parents, nb = beams(lens, W, 1, seed=7)
    ks, vs = pools_of("f16", nb, 2, 2, 64, seed=7)
    kd, vd = [x.to(DEV) for x in ks], [x.to(DEV) for x in vs]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        t = torch.from_numpy(tables).to(DEV).flatten(0, 1)
        n = torch.tensor(np.repeat(lens, W).astype(np.int32), device=DEV)
        par = torch.from_numpy(parents).to(DEV)
    pa.beam_reorder(t, n, par, kd, vd, stream=side)
    torch.cuda.synchronize()
    new, copies = B.reorder(tables, lens, parents)
    assert np.array_equal(t.cpu().numpy().reshape(tables.shape), new)
    for a, b in zip(ks + vs, kd + vd):
        assert torch.equal(bytes_of(expect(a, copies, "f16")), bytes_of(b))


def test_reorder_captured_in_place():
    """Every replay goes on from the tables that the last one left."""
    lens, W = [37, 200, 64], 4
    tables, parents, nb = beams(lens, W, 1, seed=5)
    ks, vs = pools_of("f16", nb, 2, 2, 64, seed=5)
    kd, vd = [x.to(DEV) for x in ks], [x.to(DEV) for x in vs]
    t = torch.from_numpy(tables).to(DEV).flatten(0, 1)
    n = torch.tensor(np.repeat(lens, W).astype(np.int32), device=DEV)
    par = torch.from_numpy(parents).to(DEV)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        pa.beam_reorder(t, n, par, kd, vd)
    rng = np.random.default_rng(6)
    for _ in range(6):
        parents = rng.integers(0, W, parents.shape).astype(np.int32)
        par.copy_(torch.from_numpy(parents))
        g.replay()
        torch.cuda.synchronize()
        tables, copies = B.reorder(tables, lens, parents)
        ks, vs = [expect(x, copies, "f16") for x in ks], [expect(x, copies, "f16") for x in vs]
        assert np.array_equal(t.cpu().numpy().reshape(tables.shape), tables)
        for a, b in zip(ks + vs, kd + vd):
            assert torch.equal(bytes_of(a), bytes_of(b))


# ---------------------------------------------------------------------------
# a beam search as a server runs it
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("Hq,Hkv,D,dn", [(4, 2, 64, "f16"), (4, 4, 128, "bf16")])
def test_beam_search_over_caches(Hq, Hkv, D, dn):
    """Steps of write, self attention, cross attention, selection and reordering
    over two layers, against the same search over plain contiguous states in 64
    bits that follows the device's choices; each choice is held to its own
    logits."""
    S, W, V, steps, L, dt, end = 3, 4, 501, 40, 2, DT[dn], 5
    rng = np.random.default_rng(21)
    prompt = [3, 17, 32]
    enc = [40, 0, 130]
    mb = (max(prompt) + steps) // 16 + 2
    # self-attention blocks: whole prompt blocks shared, the rest each row's own, allotted in advance
    nb = S * W * mb + 5
    perm = list(rng.permutation(nb))
    tables = np.zeros((S, W, mb), np.int32)
    for s in range(S):
        shared = prompt[s] // 16
        tables[s, :, :shared] = [perm.pop() for _ in range(shared)]
        for w in range(W):
            tables[s, w, shared:] = [perm.pop() for _ in range(mb - shared)]
    f = lambda *shape: torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(dt)    # noqa: E731
    emb_q, emb_k, emb_v = f(L, V, Hq, D), f(L, V, Hkv, D), f(L, V, Hkv, D)      # a token's projections
    pos = f(mb * 16, Hq, D) * 0.5                                                # so that steps differ
    head = torch.from_numpy((rng.standard_normal((Hq * D, V)) * 0.5).astype(np.float32))
    first = [rng.integers(0, V, n) for n in prompt]
    kc = [torch.full((nb, 16, Hkv, D), float("nan"), dtype=dt) for _ in range(L)]
    vc = [torch.full((nb, 16, Hkv, D), float("nan"), dtype=dt) for _ in range(L)]
    for l in range(L):
        for s in range(S):
            for j, tok in enumerate(first[s][:-1]):      # the last prompt token is the first step's
                blk = tables[s, 0, j // 16]
                kc[l][blk, j % 16], vc[l][blk, j % 16] = emb_k[l, tok], emb_v[l, tok]
    ek, ev = [f(24, 16, Hkv, D) for _ in range(L)], [f(24, 16, Hkv, D) for _ in range(L)]
    et = np.array([rng.permutation(24)[:9] for _ in range(S)], np.int32)
    to = lambda x: x.to(DEV)                                                     # noqa: E731
    dk, dv, dek, dev_ = [to(x) for x in kc], [to(x) for x in vc], [to(x) for x in ek], [to(x) for x in ev]
    dq, dkk, dvv, dpos, dhead = to(emb_q), to(emb_k), to(emb_v), to(pos), to(head)
    t = torch.from_numpy(tables).to(DEV).flatten(0, 1)
    det, dn_ = torch.from_numpy(et).to(DEV), torch.tensor(enc, dtype=torch.int32, device=DEV)
    lens = torch.tensor([n for n in prompt for _ in range(W)], dtype=torch.int32, device=DEV)
    scores = torch.full((S, W), -math.inf, device=DEV)
    scores[:, 0] = 0
    fin = torch.zeros((S, W), dtype=torch.uint8, device=DEV)
    tokens = torch.tensor([[first[s][-1]] * W for s in range(S)], dtype=torch.int32, device=DEV)
    scale = 1 / math.sqrt(D)
    hist = [[list(first[s]) for _ in range(W)] for s in range(S)]                # tokens of every beam
    alive = np.zeros((S, W), bool)
    alive[:, 0] = True
    for step in range(steps):
        ids = tokens.flatten().long()
        slots = pa.slot_mapping(t, lens, None, S * W, nb)
        x = torch.zeros(S * W, Hq, D, device=DEV)
        for l in range(L):
            pa.paged_kv_write(dkk[l][ids], dvv[l][ids], dk[l], dv[l], slots)
            q = dq[l][ids] + dpos[lens.long()]
            a = pa.paged_attention_decode(q, dk[l], dv[l], t, lens, scale, int(max(prompt)) + steps)
            c = pa.paged_cross_attention(q + a, dek[l], dev_[l], det, dn_, scale, max_enc_len=130)
            x = x + a.float() + c.float()
            if step % 7 == 0:                  # this layer against plain states that follow the choices
                n0 = [len(h[0]) for h in hist]
                for s in range(S):
                    for w in np.nonzero(alive[s])[0]:
                        h = torch.tensor(hist[s][w])
                        K, Vv = emb_k[l][h].double().numpy(), emb_v[l][h].double().numpy()
                        rows = -(-n0[s] // 16) * 16 - n0[s]
                        P = [np.concatenate([y, np.zeros((rows, Hkv, D))]).reshape(-1, 16, Hkv, D) for y in (K, Vv)]
                        qq = q[s * W + w:s * W + w + 1].double().cpu().numpy()
                        ref = B.cross_attention(qq, *P, np.arange(len(P[0]))[None], [n0[s]], [1], scale)
                        tol = R.bound(*ref, np.abs(Vv).max(), dt, dt)
                        got = a[s * W + w:s * W + w + 1].double().cpu().numpy()
                        assert (np.abs(got - ref[0]) <= tol).all(), (step, s, w)
                qc = (q + a).double().cpu().numpy()
                ref = B.cross_attention(qc, ek[l].double().numpy(), ev[l].double().numpy(), et, enc, [W] * S, scale)
                sel = alive.flatten()
                tol = R.bound(*ref, float(ev[l].double().abs().max()), dt, dt)
                assert (np.abs(c.double().cpu().numpy() - ref[0])[sel] <= tol[sel]).all()
        logits = (x.flatten(1) @ dhead).to(dt)
        before = scores.cpu().numpy()
        was = fin.cpu().numpy()
        got = pa.beam_select(logits, scores, W, finished=fin, end_token=end)
        check.dtype = dt
        lo = logits.view(S, W, V).cpu()
        dead = ~np.isfinite(before)
        check(got, torch.where(torch.from_numpy(dead)[..., None], torch.zeros_like(lo), lo), before, W, was, end)
        scores, parents, tokens, fin = got
        pa.beam_reorder(t, lens, parents, dk, dv)
        par, tok = parents.cpu().numpy(), tokens.cpu().numpy()
        hist = [[hist[s][par[s, w]] + [int(tok[s, w])] for w in range(W)] for s in range(S)]
        alive = np.isfinite(scores.cpu().numpy())
        lens += 1
    assert pa.device_error() == 0
