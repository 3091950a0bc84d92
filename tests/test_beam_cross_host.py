"""Host-side refusals, sizes and wrappers of cross attention and of the beam
calls (no GPU needed: a refused call reaches no CUDA call), and the references'
own checks."""
import ctypes
import math
import os

import numpy as np
import pytest
import torch

import paged_kv_attention_decode_gb300 as pa
from paged_kv_attention_decode_gb300 import _binding
from tests import _beam_ref as B
from tests._stand_in import StandIn, Stream, dev

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
F = 1 << 20          # 256-byte aligned, never dereferenced on refused calls
SIDE = 77


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_binding.library_path()):
        from paged_kv_attention_decode_gb300 import build_lib
        build_lib.build()
    return _binding.load_library()


# ---------------------------------------------------------------------------
# refusals of the library
# ---------------------------------------------------------------------------
CROSS = dict(out=F, q=F, k=F, v=F, bt=F, mb=8, n=F, cu=F, B=4, T=40, mq=20, me=100, nb=64, scale=0.1, hq=32, hkv=8,
             d=128, bs=16, ws=F, wsb=1 << 20, dt=0)


@pytest.mark.parametrize("kw,status", [
    (dict(out=None), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(bt=None), INVALID), (dict(n=None), INVALID), (dict(out=F + 8), INVALID), (dict(q=F + 2), INVALID),
    (dict(v=F + 4), INVALID), (dict(B=-1), INVALID), (dict(B=65536), INVALID), (dict(T=-1), INVALID),
    (dict(mq=-1), INVALID), (dict(me=-1), INVALID), (dict(mb=0), INVALID), (dict(mb=1 << 27), INVALID),
    (dict(nb=0), INVALID), (dict(nb=1 << 27), INVALID), (dict(scale=math.nan), INVALID),
    (dict(scale=math.inf), INVALID), (dict(hq=0), INVALID), (dict(hkv=5), INVALID), (dict(hq=520), UNSUPPORTED),
    (dict(d=96), UNSUPPORTED), (dict(bs=32), UNSUPPORTED), (dict(dt=2), UNSUPPORTED),
    (dict(cu=None, T=41), INVALID),                                     # rows that do not divide
    (dict(ws=None), WORKSPACE), (dict(wsb=100), WORKSPACE), (dict(ws=F + 16), INVALID),
    (dict(cu=None, T=40, ws=None), WORKSPACE),                          # ten rows each: chunks
    (dict(B=65535, T=65535 * 8, mq=8, hq=65535, hkv=65535, d=64), INVALID),
    (dict(T=0), 0), (dict(B=0), 0),
])
def test_cross_attention_refusals(lib, kw, status):
    assert lib.pa_paged_cross_attention(*dict(CROSS, **kw).values(), None) == status


def test_cross_workspace(lib):
    assert pa.cross_workspace_bytes(64, 512, 8) == 0 and pa.cross_workspace_bytes(0, 0, 100) == 0
    assert pa.cross_workspace_bytes(64, -1, 100) == 0
    n = pa.cross_workspace_bytes(64, 4000, 100)
    lists = 4 * (65 + 65 + 2 * (1000 + 64) + 1 + 8 * 256)
    assert lists <= n <= lists + 1024


SELECT = dict(sc=F, par=F, tok=F, fin=None, x=F, stride=200000, cum=F, ended=None, end=-1, S=2, W=4, V=200000, k=8, dt=0,
              ws=F, wsb=1 << 24)


@pytest.mark.parametrize("kw,status", [
    (dict(sc=None), INVALID), (dict(par=None), INVALID), (dict(tok=None), INVALID), (dict(x=None), INVALID),
    (dict(cum=None), INVALID), (dict(x=F + 1), INVALID), (dict(x=F + 2, dt=2), INVALID), (dict(S=-1), INVALID),
    (dict(S=65536), INVALID), (dict(W=0), INVALID), (dict(W=33), UNSUPPORTED), (dict(V=0), INVALID),
    (dict(V=(1 << 20) + 1, stride=1 << 21), UNSUPPORTED), (dict(k=0), INVALID), (dict(k=65), UNSUPPORTED),
    (dict(V=1, k=5, stride=1), INVALID), (dict(end=200000), INVALID), (dict(end=-2), INVALID), (dict(ended=F), INVALID),
    (dict(stride=199999), INVALID), (dict(dt=3), UNSUPPORTED), (dict(dt=-1), UNSUPPORTED), (dict(ws=None), WORKSPACE),
    (dict(wsb=100), WORKSPACE), (dict(ws=F + 128), INVALID), (dict(S=0), 0),
])
def test_select_refusals(lib, kw, status):
    assert lib.pa_beam_select(*dict(SELECT, **kw).values(), None) == status


def test_select_workspace(lib):
    f = lib.pa_beam_select_workspace_bytes
    for bad in ((0, 4, 100, 4, 0), (1, 33, 100, 4, 0), (1, 4, 0, 4, 0), (1, 4, (1 << 20) + 1, 4, 0), (1, 4, 100, 65, 0),
                (1, 4, 100, 4, 3), (1, 0, 100, 4, 0), (65536, 4, 100, 4, 0)):
        assert f(*bad) == 0
    # 10 numbers of 4 bytes for every 4 KB of a row
    assert f(140, 4, 32000, 8, 0) == 560 * 16 * 32 + ((560 * 16 * 8 + 255) & ~255)
    assert f(140, 4, 32000, 8, 2) > f(140, 4, 32000, 8, 1) == pa.beam_select_workspace_bytes(140, 4, 32000, 8, torch.bfloat16)
    # few requests, or small ones, need none
    assert f(1, 16, 32000, 8, 0) == f(8, 16, 32000, 64, 1) == f(32, 8, 32000, 8, 0) == f(128, 2, 32000, 2, 0) == 0
    assert f(1, 17, 32000, 8, 0) and f(9, 9, 32000, 8, 0) and f(33, 5, 32000, 8, 0) and f(65, 3, 32000, 8, 0)
    assert f(129, 1, 300, 2, 0)


PTR = ctypes.c_void_p * 2
REORDER = dict(out=F, bt=F, mb=8, n=F, par=F, S=2, W=4, k=PTR(F, F), v=PTR(F, F), L=2, nb=64, hkv=8, d=128, bs=16, kind=0)


@pytest.mark.parametrize("kw,status", [
    (dict(out=None), INVALID), (dict(bt=None), INVALID), (dict(n=None), INVALID), (dict(par=None), INVALID),
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k=PTR(F, 0)), INVALID), (dict(v=PTR(F + 8, F)), INVALID),
    (dict(S=-1), INVALID), (dict(S=65536), INVALID), (dict(W=0), INVALID), (dict(W=33), UNSUPPORTED),
    (dict(mb=0), INVALID), (dict(mb=1 << 29), INVALID), (dict(L=-1), INVALID), (dict(nb=0), INVALID),
    (dict(nb=1 << 27), INVALID), (dict(hkv=0), INVALID), (dict(d=96), UNSUPPORTED), (dict(d=64, kind=1), UNSUPPORTED),
    (dict(kind=3), UNSUPPORTED), (dict(bs=8), UNSUPPORTED),
    (dict(out=F + 4), INVALID), (dict(out=F - 2 * 4 * 8 * 4 + 4), INVALID),           # overlaps the tables
    (dict(S=0), 0),
])
def test_reorder_refusals(lib, kw, status):
    assert lib.pa_beam_reorder(*dict(REORDER, **kw).values(), None) == status


# ---------------------------------------------------------------------------
# the wrappers
# ---------------------------------------------------------------------------
def z(*shape, dtype=torch.float16):
    return dev(torch.zeros(shape, dtype=dtype))


I32, F32 = torch.int32, torch.float32


def cross_args(**kw):
    a = dict(q=z(12, 8, 64), k_cache=z(9, 16, 2, 64), v_cache=z(9, 16, 2, 64), block_tables=z(3, 4, dtype=I32),
             enc_lens=z(3, dtype=I32), scale=0.1, max_enc_len=30)
    return dict(a, **kw)


def select_args(**kw):
    return dict(dict(logits=z(6, 100), scores=z(2, 3, dtype=F32), num_out=4), **kw)


def reorder_args(**kw):
    a = dict(block_tables=z(6, 5, dtype=I32), seq_lens=z(6, dtype=I32), parents=z(2, 3, dtype=I32),
             k_caches=[z(9, 16, 2, 64), z(9, 16, 2, 64)], v_caches=[z(9, 16, 2, 64), z(9, 16, 2, 64)])
    return dict(a, **kw)


CALLS = {"cross": (pa.paged_cross_attention, cross_args), "select": (pa.beam_select, select_args),
         "reorder": (pa.beam_reorder, reorder_args)}


@pytest.mark.parametrize("name,kw,msg", [
    ("cross", dict(q=z(13, 8, 64)), "same number of rows"), ("cross", dict(enc_lens=z(0, dtype=I32)), "same number"),
    ("cross", dict(q=z(12, 8, 128)), "cache"), ("cross", dict(v_cache=z(9, 16, 2, 64, dtype=torch.bfloat16)), "cache"),
    ("cross", dict(block_tables=z(2, 4, dtype=I32)), "table"), ("cross", dict(enc_lens=z(3, dtype=torch.int64)), "int32"),
    ("cross", dict(cu_q_lens=z(3, dtype=I32), max_q_len=4), "cu_q_lens"), ("cross", dict(out=z(12, 8, 32)), "out"),
    ("cross", dict(q=torch.zeros(12, 8, 64, dtype=torch.float16)), None),
    ("cross", dict(q=z(12, 8, 128)[..., ::2]), "contiguous"),
    ("select", dict(logits=z(5, 100)), "logits"), ("select", dict(logits=z(6, 200)[:, ::2]), "logits"),
    ("select", dict(logits=z(6, 100, dtype=torch.float64)), "dtype"), ("select", dict(scores=z(2, 3)), "scores"),
    ("select", dict(num_out=0), "num_out"), ("select", dict(logits=z(2, 4, 100)[:, :3].transpose(0, 1)), "logits"),
    ("select", dict(finished=z(2, 3, dtype=I32), end_token=1), "finished"),
    ("select", dict(finished=z(2, 3, dtype=torch.uint8)), "end_token"),
    ("select", dict(finished=z(2, 3, dtype=torch.uint8), end_token=100), "end_token"),
    ("select", dict(out=(z(2, 4, dtype=F32), z(2, 4, dtype=I32))), "out"),
    ("select", dict(out=(z(2, 4, dtype=F32), z(2, 4, dtype=I32), z(2, 4, dtype=torch.int64))), "out"),
    ("select", dict(logits=torch.zeros(6, 100)), None),
    ("reorder", dict(block_tables=z(5, 5, dtype=I32)), "block_tables"),
    ("reorder", dict(block_tables=z(6, 5, dtype=torch.int64)), "block_tables"),
    ("reorder", dict(seq_lens=z(2, dtype=I32)), "seq_lens"), ("reorder", dict(parents=z(2, 3, dtype=torch.int64)), "parents"),
    ("reorder", dict(k_caches=[z(9, 16, 2, 64)]), "caches"), ("reorder", dict(v_caches=[z(9, 16, 2, 64), z(8, 16, 2, 64)]), "caches"),
    ("reorder", dict(k_caches=[z(9, 2, 2, 64)] * 2), "pools"), ("reorder", dict(out=z(6, 4, dtype=I32)), "out"),
    ("reorder", dict(k_caches=[z(9, 16, 2, 128)[..., ::2]] * 2), "caches"),
])
def test_wrappers_refuse(monkeypatch, name, kw, msg):
    s = StandIn(monkeypatch)
    call, args = CALLS[name]
    with pytest.raises((pa.PagedAttnError, RuntimeError), match=msg):
        call(**args(**kw))
    assert not s.calls


def test_wrappers_pass_sizes(monkeypatch):
    s = StandIn(monkeypatch)
    pa.paged_cross_attention(**cross_args())
    (name, a), = s.calls
    assert name == "pa_paged_cross_attention" and a[7] is None and a[8:13] == (3, 12, 4, 30, 9) and a[18:20] == (None, 0)
    s.calls.clear()
    pa.paged_cross_attention(**cross_args(q=z(30, 8, 64), cu_q_lens=z(4, dtype=I32), max_q_len=20))
    a = s.calls[0][1]
    assert a[7] is not None and a[8:11] == (3, 30, 20) and a[18] is not None and a[19] == 4096
    s.calls.clear()
    # three dimensions, strided rows, one beam, one request
    for x, stride in ((z(2, 3, 100), 100), (z(2, 3, 120)[..., :100], 120), (z(6, 100), 100)):
        pa.beam_select(**select_args(logits=x))
        a = s.calls.pop()[1]
        assert a[5] == stride and a[9:14] == (2, 3, 100, 4, 0) and a[3] is None
    for S, W, x in ((1, 3, z(2, 3, 100)[:1]), (3, 1, z(3, 5, 100)[:, :1])):
        pa.beam_select(x, z(S, W, dtype=F32), 4)
        a = s.calls.pop()[1]
        assert a[5] == x.stride(1 if S == 1 else 0) and a[9:11] == (S, W)
    got = pa.beam_select(**select_args(finished=z(2, 3, dtype=torch.bool), end_token=7))
    assert [t.dtype for t in got] == [F32, I32, I32, torch.bool] and s.calls.pop()[1][8] == 7
    for k, kind in (([z(9, 16, 2, 64)], 0), ([z(9, 2, 16, 128, dtype=torch.uint8)], 1),
                    ([z(9, 2, 576, dtype=torch.uint8)], 2)):
        args = reorder_args(k_caches=k[0], v_caches=k)                  # a pool, or a list of them
        assert pa.beam_reorder(**args) is args["block_tables"]
        a = s.calls.pop()[1]
        assert a[0] == a[1] and a[9:15] == (1, 9, 2, 128 if kind == 1 else 64, 16, kind)
    out = z(6, 5, dtype=I32)
    assert pa.beam_reorder(**reorder_args(k_caches=[], v_caches=[], out=out)) is out


@pytest.mark.parametrize("as_handle", [False, True])
@pytest.mark.parametrize("name", ["cross", "select", "reorder"])
def test_a_given_stream_owns_what_the_call_makes(monkeypatch, name, as_handle):
    s = StandIn(monkeypatch)
    call, args = CALLS[name]
    a = args()
    s.made.clear()
    out = call(**a, stream=SIDE if as_handle else Stream(SIDE))
    assert {h for _, _, h in s.made} <= {SIDE} and (s.made or name == "reorder")
    assert s.calls[0][1][-1] == SIDE and s.now.cuda_stream == 0
    for t in out if isinstance(out, tuple) else (out,):
        assert getattr(t, "recorded", None) == (None if name == "reorder" else [0])


def test_given_results_stay_the_callers(monkeypatch):
    s = StandIn(monkeypatch)
    out = (z(2, 4, dtype=F32), z(2, 4, dtype=I32), z(2, 4, dtype=I32))
    ws = z(8192, dtype=torch.uint8)
    s.made.clear()
    got = pa.beam_select(**select_args(out=out, workspace=ws, stream=Stream(SIDE)))
    assert all(a is b for a, b in zip(got, out)) and not s.made
    assert not any(hasattr(t, "recorded") for t in out)


# ---------------------------------------------------------------------------
# the references
# ---------------------------------------------------------------------------
def test_reference_cross_attention_is_attention_without_a_mask():
    rng = np.random.default_rng(0)
    lens, qlens, Hq, H, D = [40, 0, 5], [3, 2, 7], 4, 2, 8
    kp, vp = rng.standard_normal((6, 16, H, D)), rng.standard_normal((6, 16, H, D))
    tables = np.array([[3, 0, 5], [1, 1, 1], [4, 0, 0]])
    q = rng.standard_normal((12, Hq, D))
    out, A, smax, n = B.cross_attention(q, kp, vp, tables, lens, qlens, 0.3)
    r = 0
    for b, (m, c) in enumerate(zip(lens, qlens)):
        if m:
            k = torch.from_numpy(kp[tables[b]].reshape(-1, H, D)[:m]).transpose(0, 1).repeat_interleave(2, 0)
            v = torch.from_numpy(vp[tables[b]].reshape(-1, H, D)[:m]).transpose(0, 1).repeat_interleave(2, 0)
            ref = torch.nn.functional.scaled_dot_product_attention(torch.from_numpy(q[r:r + c]).transpose(0, 1), k, v, scale=0.3)
            assert np.allclose(out[r:r + c], ref.transpose(0, 1).numpy(), atol=1e-12)
        else:
            assert not out[r:r + c].any()
        r += c
    assert (A >= np.abs(out) - 1e-12).all() and smax.shape == n.shape == (12, Hq, 1)


def test_reference_selection_by_hand():
    ln = math.log
    x = np.log(np.array([[[1., 1, 2], [3, 1, 4]], [[1, 1, 1], [1, 1, 1]]]))
    cum = np.array([[ln(0.5), ln(0.8)], [0.0, -np.inf]], np.float32)
    sc, par, tok, fin = B.select(x, cum, 4)
    # 0.125 0.125 0.25 | 0.3 0.1 0.4
    assert np.allclose(np.exp(sc[0]), [0.4, 0.3, 0.25, 0.125], atol=1e-6)
    assert par[0].tolist() == [1, 1, 0, 0] and tok[0].tolist() == [2, 0, 2, 0]
    assert par[1].tolist() == [0, 0, 0, 1] and tok[1].tolist() == [0, 1, 2, 0] and np.isneginf(sc[1, 3])
    ended = np.array([[0, 1], [1, 0]])
    sc, par, tok, fin = B.select(x, cum, 2, ended, 1)
    assert np.allclose(np.exp(sc[0]), [0.8, 0.25], atol=1e-6) and par[0].tolist() == [1, 0] and tok[0].tolist() == [1, 2]
    assert fin.tolist() == [[True, False], [True, True]]         # (the filler's parent had ended)
    x[0, 0, 0], x[0, 1, 2] = np.nan, np.inf
    sc, par, tok, _ = B.select(x[:1], cum[:1], 2, top=100.0)
    assert (par[0, 0], tok[0, 0]) == (1, 2) and (par[0, 1], tok[0, 1]) == (0, 2)
    assert np.allclose(np.exp(sc[0]), [0.8, 0.5 * 2 / 3])


@pytest.mark.parametrize("n", [0, 7, 16, 40, 95])
def test_reference_reordering_keeps_every_history(n):
    """Row j's tokens are what its parent's were, and no two rows end in one block."""
    rng = np.random.default_rng(n)
    W, mb = 5, 6
    perm = rng.permutation(W * mb + 2)
    tables = np.stack([np.concatenate([perm[:1], perm[2 + w * (mb - 1):2 + (w + 1) * (mb - 1)]]) for w in range(W)])[None]
    if n < 16:                                      # (a last block that rows share is no valid input)
        tables[0] = perm[:W * mb].reshape(W, mb)
    pool = rng.integers(0, 1000, (W * mb + 2, 16))
    parents = rng.integers(0, W, (1, W))

    def history(t, p):
        return [p[t[0, w, np.arange(n) // 16], np.arange(n) % 16] for w in range(W)]

    before = history(tables, pool)
    new, copies = B.reorder(tables, [n], parents)
    after = pool.copy()
    for src, dst, t in copies:
        assert src != dst
        after[dst, :t] = pool[src, :t]
    for w, h in enumerate(history(new, after)):
        assert np.array_equal(h, before[parents[0, w]])
    if n % 16:
        assert len(set(new[0, :, n // 16])) == W
    assert np.array_equal(new[0, :, n // 16 + 1:], tables[0, :, n // 16 + 1:])
    assert set(new[0].ravel()) <= set(tables[0].ravel())
