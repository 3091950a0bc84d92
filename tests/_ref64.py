"""Plain 64-bit references of the append, 4-bit cache and modified-score
attention operators, with the error bounds the tests hold the kernels to.

Nothing here imports the product package.
"""
import math

import numpy as np
import torch

# half a step of each type, relative to the value
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
SUB = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}   # half a subnormal step
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=np.float64)


def e4m3_table():
    t = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        if (c & 127) == 127:
            v = math.nan
        t[c] = -v if c & 128 else v
    return t


E4M3 = e4m3_table()


def rope32(x, cos_sin, pos, rot, interleaved):
    """The rotation's definition in fp32 steps: x [T, H, D] float32 numpy."""
    x = x.astype(np.float32)
    half = rot // 2
    c = cos_sin[pos][:, None, :half].astype(np.float32)
    s = cos_sin[pos][:, None, half:].astype(np.float32)
    ia, ib = (np.arange(0, rot, 2), np.arange(1, rot, 2)) if interleaved else (np.arange(half), np.arange(half, rot))
    y = x.copy()
    y[..., ia] = (x[..., ia] * c) - (x[..., ib] * s)
    y[..., ib] = (x[..., ib] * c) + (x[..., ia] * s)
    return y


def rope64(x, cos_sin, pos, rot, interleaved):
    """The rotation in 64 bits, and |a cos| + |b sin| per element (for the bound)."""
    x = x.astype(np.float64)
    half = rot // 2
    c, s = cos_sin[pos][:, None, :half].astype(np.float64), cos_sin[pos][:, None, half:].astype(np.float64)
    ia, ib = (np.arange(0, rot, 2), np.arange(1, rot, 2)) if interleaved else (np.arange(half), np.arange(half, rot))
    y, mag = x.copy(), np.abs(x)
    y[..., ia], y[..., ib] = x[..., ia] * c - x[..., ib] * s, x[..., ib] * c + x[..., ia] * s
    mag[..., ia] = np.abs(x[..., ia] * c) + np.abs(x[..., ib] * s)
    mag[..., ib] = np.abs(x[..., ib] * c) + np.abs(x[..., ia] * s)
    return y, mag


def nearest_even(x, grid):
    """Index of the nearest value of the ascending grid to each x >= 0 (ties to
    the even index, past the end the last)."""
    x = np.minimum(x, grid[-1])
    hi = np.minimum(np.searchsorted(grid, x), len(grid) - 1)
    lo = np.maximum(hi - 1, 0)
    up, down = grid[hi] - x, x - grid[lo]
    return np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)


def quantise_fp4(x, scale):
    """x [..., D] float32 -> (codes [..., D], scale codes [..., D / 16]) by the
    definition: fp32 product with 1 / scale, fp32 quotients, ties to even."""
    inv = np.float32(1.0) / np.float32(scale)
    y = (x.astype(np.float32) * inv).astype(np.float32)
    g = y.reshape(*y.shape[:-1], -1, 16)
    mx = np.abs(g).max(-1)                                 # (NaN stays NaN)
    nan = np.isnan(mx)
    with np.errstate(all="ignore"):
        u = (mx / np.float32(6.0)).astype(np.float32)
    sc = nearest_even(np.where(nan, 0, u).astype(np.float64), E4M3[:127])
    sv = E4M3[sc].astype(np.float32)[..., None]
    live = (sv > 0) & ~nan[..., None]
    with np.errstate(all="ignore"):
        q = np.where(live, g / np.where(live, sv, np.float32(1)), np.float32(0)).astype(np.float32)
    codes = nearest_even(np.abs(q).astype(np.float64), E2M1[:8]) | (np.signbit(q) << 3)
    sc = np.where(nan, 127, sc)
    return codes.reshape(x.shape).astype(np.uint8), sc.astype(np.uint8)


def pack_tiles(codes, scales, v):
    """Token-major blocks (codes [NB, 16, H, D], scales [NB, 16, H, D / 16]) -> tiles [NB, H, 9 D]."""
    NB, _, H, D = codes.shape
    body = (codes[..., 0::2] | (codes[..., 1::2] << 4)).transpose(0, 2, 1, 3).reshape(NB, H, -1)
    s = scales.transpose(0, 2, 3, 1) if v else scales.transpose(0, 2, 1, 3)
    return np.concatenate([body, s.reshape(NB, H, -1)], -1).astype(np.uint8)


def unpack_tiles(tiles, v):
    """Tiles [NB, H, 9 D] -> codes [NB, 16, H, D], scale codes [NB, 16, H, D / 16]."""
    NB, H, n = tiles.shape
    D = n // 9
    body = tiles[..., :8 * D].reshape(NB, H, 16, D // 2)
    codes = np.stack([body & 15, body >> 4], -1).reshape(NB, H, 16, D).transpose(0, 2, 1, 3)
    s = tiles[..., 8 * D:]
    s = s.reshape(NB, H, D // 16, 16).transpose(0, 3, 1, 2) if v else s.reshape(NB, H, 16, D // 16).transpose(0, 2, 1, 3)
    return codes, s


def tile_values(tiles, v, scale=1.0):
    """Values of tiles, token-major [NB, 16, H, D], in 64 bits."""
    codes, s = unpack_tiles(tiles, v)
    return E2M1[codes] * np.repeat(E4M3[s], 16, -1) * scale


def attention(q, k_pool, v_pool, tables, lens, qlens, scale, softcap=0.0, window=0, slopes=None, bad=()):
    """Attention of every query row over token-major 64-bit pools [NB, 16, H, D].
    q [T, Hq, D].  `bad`: physical ids whose tokens contribute nothing.
    Returns (out, A, smax, n): A = sum of p |v| per output element, smax = the
    largest sum of |q_d k_d| scale of a row, n = its visible keys (for the bound)."""
    T, Hq, D = q.shape
    NB, _, H, _ = k_pool.shape
    G = Hq // H
    out, A = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    smax, cnt = np.zeros((T, Hq, 1)), np.ones((T, Hq, 1))
    r = 0
    for b, (n, c) in enumerate(zip(lens, qlens)):
        n, c = int(n), int(c)
        for i in range(c):
            pos = n - c + i
            lo = max(0, pos - window + 1) if window else 0
            j = np.arange(lo, pos + 1)
            ids = tables[b, j // 16].astype(np.int64)
            ok = (ids >= 0) & (ids < NB) & ~np.isin(ids, list(bad))
            j, ids = j[ok], ids[ok]
            if n > 0 and len(j):
                k, v = k_pool[ids, j % 16], v_pool[ids, j % 16]           # [n, H, D]
                qq = q[r].reshape(H, G, D)
                s = np.einsum("hgd,nhd->hgn", qq, k) * scale
                mag = np.einsum("hgd,nhd->hgn", np.abs(qq), np.abs(k)) * abs(scale)
                if softcap:
                    s = softcap * np.tanh(s / softcap)
                if slopes is not None:
                    s = s + slopes.reshape(H, G, 1) * (j - pos)
                p = np.exp(s - s.max(-1, keepdims=True))
                p /= p.sum(-1, keepdims=True)
                out[r] = np.einsum("hgn,nhd->hgd", p, v).reshape(Hq, D)
                A[r] = np.einsum("hgn,nhd->hgd", p, np.abs(v)).reshape(Hq, D)
                smax[r] = mag.max(-1).reshape(Hq, 1)
                cnt[r] = len(j)
            r += 1
    return out, A, smax, cnt


def bound(out, A, smax, cnt, vmax, dtype, p_dtype, softcap=0.0, bias=0.0):
    """How far a kernel's output may be from `out`:
      * the output's own rounding: U |out| (and a subnormal step);
      * the weights, rounded to p_dtype before the product with V: U A; fp16
        weights below 2^-14 of the row's reference are subnormal: 2^-25 vmax
        each (the softmax sum is at least 1);
      * scores: fp32 sums of D <= 128 products and a few steps more, each 2^-24
        of smax (`d` below, in natural units); tanh through 2^x and a
        reciprocal, each a few ulp of 1: 2^-21 of the cap; the distance bias
        2^-22 of `bias`; 2^x itself 2^-21.  An error d of a score moves the
        output by at most 2 d A (numerator and sum)."""
    d = 140 * 2.0 ** -24 * smax + 2.0 ** -21 * softcap + 2.0 ** -22 * bias + 2.0 ** -20
    sub = SUB[p_dtype] * cnt * vmax
    return U[dtype] * np.abs(out) + SUB[dtype] + (U[p_dtype] + 2 * d + 2.0 ** -20) * A * (1 + U[dtype]) + 2 * sub
