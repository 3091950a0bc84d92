"""Plain 64-bit references of cross attention, beam selection and beam
reordering.  Nothing here imports the product package."""
import math

import numpy as np

BS = 16


def cross_attention(q, k_pool, v_pool, tables, lens, qlens, scale):
    """q [T, Hq, D], token-major 64-bit pools [NB, 16, H, D]; every row of a
    sequence sees all its states (blocks outside the pool contribute nothing).
    Returns (out, A, smax, n) as `_ref64.attention` does, for its `bound`."""
    T, Hq, D = q.shape
    NB, _, H, _ = k_pool.shape
    G = Hq // H
    out, A = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    smax, cnt = np.zeros((T, Hq, 1)), np.ones((T, Hq, 1))
    r = 0
    for b, (n, c) in enumerate(zip(lens, qlens)):
        n, c = int(n), int(c)
        j = np.arange(n)
        ids = tables[b, j // BS].astype(np.int64)
        ok = (ids >= 0) & (ids < NB)
        j, ids = j[ok], ids[ok]
        if c and len(j):
            k, v = k_pool[ids, j % BS], v_pool[ids, j % BS]          # [n, H, D]
            qq = q[r:r + c].reshape(c, H, G, D)
            s = np.einsum("chgd,nhd->chgn", qq, k) * scale
            mag = np.einsum("chgd,nhd->chgn", np.abs(qq), np.abs(k)) * abs(scale)
            p = np.exp(s - s.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            out[r:r + c] = np.einsum("chgn,nhd->chgd", p, v).reshape(c, Hq, D)
            A[r:r + c] = np.einsum("chgn,nhd->chgd", p, np.abs(v)).reshape(c, Hq, D)
            smax[r:r + c] = mag.max(-1).reshape(c, Hq, 1)
            cnt[r:r + c] = len(j)
        r += c
    return out, A, smax, cnt


def candidate_scores(logits, scores, finished=None, end_token=-1, top=None):
    """Scores of every candidate [S, W, V] in 64 bits.  logits [S, W, V]; `top` is
    the logits' type's largest value."""
    S, W, V = logits.shape
    x = np.where(np.isnan(logits), -np.inf, logits.astype(np.float64))
    if top is not None:
        x = np.minimum(x, top)
    cum = np.where(np.isnan(scores), -np.inf, scores.astype(np.float64))
    cum = np.minimum(cum, float(np.finfo(np.float32).max))
    out = np.full((S, W, V), -np.inf)
    for s in range(S):
        for w in range(W):
            if cum[s, w] == -np.inf:
                continue
            if finished is not None and finished[s, w]:
                out[s, w, end_token] = cum[s, w]
                continue
            m = x[s, w].max()
            if m > -np.inf:
                e = np.exp(x[s, w] - m)
                lse = math.log(math.fsum(e)) if V <= 4096 else math.log(e.sum())
                out[s, w] = cum[s, w] + (x[s, w] - m - lse)
    out[out < -float(np.finfo(np.float32).max)] = -np.inf
    return out


def select(logits, scores, k, finished=None, end_token=-1, top=None):
    """(scores, parents, tokens, finished) [S, k] of the k best candidates, ties to
    the lowest w V + v.  (Beside a score so large that 64 bits swallow a log
    probability, 3e38 say, what they swallow still orders the candidates.)"""
    S, W, V = logits.shape
    c = candidate_scores(logits, scores, finished, end_token, top).reshape(S, W * V)
    cum = np.nan_to_num(scores.astype(np.float64), nan=0.0, posinf=float(np.finfo(np.float32).max), neginf=0.0)
    lp = candidate_scores(logits, np.where(scores > -np.inf, 0.0, scores), finished, end_token, top).reshape(S, W * V)
    with np.errstate(invalid="ignore"):
        big = np.repeat(np.abs(cum), V, 1) > 2.0 ** 60
        rest = np.where(big & np.isfinite(c), lp, 0.0)
    at = np.stack([np.lexsort((np.arange(W * V), -rest[s], -c[s]))[:k] for s in range(S)])
    parents, tokens = at // V, at % V
    fin = np.zeros((S, W), bool) if finished is None else finished.astype(bool)
    return (np.take_along_axis(c, at, 1), parents, tokens,
            np.take_along_axis(fin, parents, 1) | (tokens == end_token))


def reorder(tables, lens, parents):
    """tables [S, W, max_blocks], lens [S], parents [S, W] -> (new tables, copies
    (source block, destination block, tokens))."""
    new, copies = tables.copy(), []
    for s, n in enumerate(lens):
        f, t = divmod(int(n), BS)
        taken = set()
        spare = [tables[s, p, f] for p in range(tables.shape[1]) if p not in parents[s]] if t else []
        for j, p in enumerate(parents[s]):
            new[s, j, :f] = tables[s, p, :f]
            if not t:
                continue
            if p not in taken:
                taken.add(p)
                new[s, j, f] = tables[s, p, f]
            else:
                new[s, j, f] = spare.pop(0)
                copies.append((int(tables[s, p, f]), int(new[s, j, f]), t))
    return new, copies
