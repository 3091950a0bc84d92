"""Host-side refusals and sizes of the rotate-and-append, 4-bit cache and
modified-score calls (no GPU needed: a refused call reaches no CUDA call), and
the references' own checks."""
import ctypes
import math

import numpy as np
import pytest
import torch

import paged_kv_attention_decode_gb300 as pa
from paged_kv_attention_decode_gb300 import _binding
from tests import _ref64 as R

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
F = 1 << 20          # 256-byte aligned, never dereferenced on refused calls


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(_binding.library_path()):
        from paged_kv_attention_decode_gb300 import build_lib
        build_lib.build()
    return _binding.load_library()


ROPE = dict(q_out=F, qos=4096, q=F, qs=4096, key=F, ks=1024, value=F, vs=1024, kc=F, vc=F, slots=F, pos=F, table=F,
            maxp=100, T=4, nb=8, hq=32, hkv=8, d=128, rot=128, inter=0, bs=16, dt=0)


@pytest.mark.parametrize("name", ["pa_paged_rope_kv_write", "pa_paged_rope_kv_write_fp8",
                                  "pa_paged_rope_kv_write_fp4"])
@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(q_out=None), INVALID), (dict(key=None), INVALID), (dict(value=None), INVALID),
    (dict(kc=None), INVALID), (dict(slots=None), INVALID), (dict(pos=None), INVALID), (dict(table=None), INVALID),
    (dict(q=F + 2), INVALID), (dict(key=F + 8), INVALID), (dict(vc=F + 4), INVALID), (dict(table=F + 4), INVALID),
    (dict(T=-1), INVALID), (dict(nb=0), INVALID), (dict(hkv=0), INVALID), (dict(hq=-1), INVALID),
    (dict(rot=0), INVALID), (dict(rot=144), INVALID), (dict(rot=24), UNSUPPORTED), (dict(inter=2), INVALID),
    (dict(maxp=0), INVALID), (dict(d=96, rot=96), UNSUPPORTED), (dict(bs=32), UNSUPPORTED),
    (dict(dt=2), UNSUPPORTED), (dict(qs=4092), INVALID), (dict(qs=4100), UNSUPPORTED), (dict(ks=1020), INVALID),
    (dict(vs=0), INVALID), (dict(qos=8192), INVALID),          # in place with another stride
])
def test_rope_append_refusals(lib, name, kw, status):
    a = dict(ROPE, **kw)
    args = list(a.values())
    if name != "pa_paged_rope_kv_write":
        args += [0.5, 0.5]
    assert getattr(lib, name)(*args, None) == status


@pytest.mark.parametrize("ks,vs", [(0.0, 1.0), (1.0, -1.0), (math.nan, 1.0), (1.0, math.inf), (1e-45, 1.0)])
def test_quantised_append_refuses_scales(lib, ks, vs):
    assert lib.pa_paged_rope_kv_write_fp8(*ROPE.values(), ks, vs, None) == INVALID
    assert lib.pa_paged_rope_kv_write_fp4(*ROPE.values(), ks, vs, None) == INVALID
    assert lib.pa_paged_kv_write_fp4(F, F, F, F, F, 4, 8, 8, 128, 16, 0, ks, vs, None) == INVALID


def test_fp8_append_takes_head_dim_128_only(lib):
    a = dict(ROPE, d=64, rot=64, qs=2048, qos=2048, ks=512, vs=512)
    assert lib.pa_paged_rope_kv_write_fp8(*a.values(), 0.5, 0.5, None) == UNSUPPORTED


def test_fp4_write_and_unpack_refusals(lib):
    w = lib.pa_paged_kv_write_fp4
    assert w(None, F, F, F, F, 4, 8, 8, 128, 16, 0, 1.0, 1.0, None) == INVALID
    assert w(F, F, F, F + 8, F, 4, 8, 8, 128, 16, 0, 1.0, 1.0, None) == INVALID
    assert w(F, F, F, F, F, 4, 8, 8, 96, 16, 0, 1.0, 1.0, None) == UNSUPPORTED
    assert w(F, F, F, F, F, 4, 8, 8, 128, 8, 0, 1.0, 1.0, None) == UNSUPPORTED
    assert w(F, F, F, F, F, 0, 8, 8, 128, 16, 0, 1.0, 1.0, None) == 0
    u = lib.pa_paged_kv_unpack_fp4
    assert u(None, F, F, F, 8, 8, 128, 16, 1.0, 1.0, 0, None) == INVALID
    assert u(F, F, F, F + 4, 8, 8, 128, 16, 1.0, 1.0, 0, None) == INVALID
    assert u(F, F, F, F, -1, 8, 128, 16, 1.0, 1.0, 0, None) == INVALID
    assert u(F, F, F, F, 8, 8, 32, 16, 1.0, 1.0, 0, None) == UNSUPPORTED
    assert u(F, F, F, F, 8, 8, 128, 16, math.nan, 1.0, 0, None) == INVALID
    assert u(F, F, F, F, 0, 8, 128, 16, 1.0, 1.0, 0, None) == 0


DEC = dict(out=F, q=F, kc=F, vc=F, bt=F, mb=64, sl=F, B=4, ml=1000, nb=300, scale=0.1)
VAR = dict(out=F, q=F, kc=F, vc=F, bt=F, mb=64, sl=F, cu=F, B=4, T=100, mq=97, ml=1000, nb=300, scale=0.1)
TAIL = dict(hq=32, hkv=8, d=128, bs=16, part=0, ws=F, wsb=1 << 40, dt=0)


def call(lib, kind, cache, **kw):
    a = dict(DEC if kind == "decode" else VAR)
    a.update(dict(k_scale=1.0, v_scale=1.0) if cache == "fp4" else dict(softcap=0.0, window=0, slopes=None))
    a.update(TAIL)
    if kind != "decode":
        del a["part"]
    a.update(kw)
    return getattr(lib, f"pa_paged_attention_{kind}_{cache}")(*a.values(), None)


@pytest.mark.parametrize("kind", ["decode", "prefill"])
@pytest.mark.parametrize("cache", ["fp4", "mod"])
@pytest.mark.parametrize("kw,status", [
    (dict(out=None), INVALID), (dict(q=F + 8), INVALID), (dict(kc=F + 2), INVALID), (dict(bt=None), INVALID),
    (dict(sl=None), INVALID), (dict(B=-1), INVALID), (dict(ml=-1), INVALID), (dict(mb=0), INVALID),
    (dict(nb=0), INVALID), (dict(scale=math.inf), INVALID), (dict(hq=33), INVALID), (dict(hkv=0), INVALID),
    (dict(hq=8 * 65), UNSUPPORTED), (dict(d=96), UNSUPPORTED), (dict(bs=32), UNSUPPORTED), (dict(dt=3), UNSUPPORTED),
    (dict(ws=None), WORKSPACE), (dict(wsb=100), WORKSPACE), (dict(ws=F + 16), INVALID),
])
def test_attention_refusals(lib, kind, cache, kw, status):
    assert call(lib, kind, cache, **kw) == status


@pytest.mark.parametrize("kind", ["decode", "prefill"])
def test_attention_refuses_scales_and_modifications(lib, kind):
    assert call(lib, kind, "fp4", k_scale=math.nan) == INVALID
    assert call(lib, kind, "fp4", v_scale=math.inf) == INVALID
    for bad in (dict(softcap=-1.0), dict(softcap=math.nan), dict(softcap=1000.5), dict(softcap=1e-40),
                dict(window=-1)):
        assert call(lib, kind, "mod", **bad) == INVALID
    assert call(lib, kind, "mod", B=0) == 0
    assert call(lib, kind, "fp4", B=0) == 0


def test_decode_partition_argument(lib):
    assert call(lib, "decode", "fp4", part=24) == INVALID
    assert call(lib, "decode", "mod", part=-16) == INVALID


@pytest.mark.parametrize("cache", ["fp4", "mod"])
def test_too_many_work_items_are_refused(lib, cache):
    assert call(lib, "decode", cache, B=60000, ml=1000000, part=64, hq=16, hkv=16) == INVALID
    assert call(lib, "prefill", cache, T=2 ** 31 - 1, hq=16, hkv=16, mq=2048) == INVALID


def test_partition_for(lib):
    assert pa.decode_partition_for(64, 32, 32, 4096) == 512       # plenty of items
    assert pa.decode_partition_for(8, 64, 8, 131072) == 2048      # exactly 4096 items
    assert pa.decode_partition_for(8, 64, 8, 120000) == 1024
    assert pa.decode_partition_for(3, 8, 8, 700) == 64
    assert pa.decode_partition_for(1, 32, 32, 4096) == 128        # 64 < sqrt(8192)
    assert pa.decode_partition_for(4, 4, 4, 128) == 512           # one partition
    assert pa.decode_partition_for(0, 4, 4, 4096) == 128
    for bad in ((-1, 4, 4, 10), (1, 0, 4, 10), (1, 4, 0, 10), (1, 4, 3, 10), (1, 4, 4, -1)):
        with pytest.raises(pa.PagedAttnError):
            pa.decode_partition_for(*bad)
    for args in ((1, 32, 8, 1000), (64, 64, 8, 100000), (2, 8, 1, 77)):
        assert pa.decode_partition_for(*args) <= pa.decode_partition(args[3]) and \
            pa.decode_partition_for(*args) % 16 == 0


def test_workspace_sizes(lib):
    # the same call with the automatic partition is never smaller than the plain one's
    assert pa.prefill_mod_workspace_bytes(4, 100, 32, 8, 128, 1000) >= pa.prefill_workspace_bytes(4, 100, 32, 128, 1000)
    # many sequences: the same partition, the same size
    assert pa.prefill_mod_workspace_bytes(600, 600, 32, 8, 128, 4096) == \
        pa.prefill_workspace_bytes(600, 600, 32, 128, 4096)
    mod = pa.prefill_mod_workspace_bytes(4, 100, 32, 8, 128, 1000)
    per = 2 * 16 * 8 * 128 * 2
    copy = pa.prefill_fp4_workspace_bytes(4, 100, 32, 8, 128, 1000, 64, 1000) - mod
    assert (63 + 4) * per <= copy <= (63 + 4) * per + 4096
    assert pa.prefill_mod_workspace_bytes(4, 100, 32, 5, 128, 1000) == 0
    assert pa.prefill_fp4_workspace_bytes(4, 100, 32, 8, 128, 1000, 0, 10) == 0
    need = pa.prefill_mod_workspace_bytes(4, 100, 32, 8, 128, 1000)
    assert call(lib, "prefill", "mod", wsb=need - 1) == WORKSPACE
    assert call(lib, "prefill", "fp4", wsb=need) == WORKSPACE      # a chunk needs room for its copy


def test_tile_bytes(lib):
    assert pa.fp4_tile_bytes(128) == 1152 and pa.fp4_tile_bytes(64) == 576
    with pytest.raises(pa.PagedAttnError):
        pa.fp4_tile_bytes(96)


def test_bindings_refuse_cpu_tensors_and_shapes(lib):
    if not torch.cuda.is_available():
        q = torch.zeros(2, 8, 128, dtype=torch.float16)
        with pytest.raises((pa.PagedAttnError, RuntimeError, AssertionError)):
            pa.paged_attention_decode_mod(q, torch.zeros(4, 16, 8, 128, dtype=torch.float16),
                                          torch.zeros(4, 16, 8, 128, dtype=torch.float16),
                                          torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), 0.1, 10)
    with pytest.raises(pa.PagedAttnError):
        pa.paged_kv_write_fp4(torch.zeros(2, 8, 96), torch.zeros(2, 8, 96), torch.zeros(4, 8, 864, dtype=torch.uint8),
                              torch.zeros(4, 8, 864, dtype=torch.uint8), torch.zeros(2, dtype=torch.int64), 1.0, 1.0)


# ---- the references themselves ---------------------------------------------

def test_reference_e4m3_matches_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    t = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(t), np.isnan(R.E4M3)) and np.array_equal(t[~np.isnan(t)], R.E4M3[~np.isnan(t)])
    x = np.concatenate([np.linspace(0, 500, 4001), [0.0009765625, 0.0029296875, 432, 464]]).astype(np.float32)
    want = torch.from_numpy(np.minimum(x, 448)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(R.nearest_even(x.astype(np.float64), R.E4M3[:127]), want)


def test_reference_quantiser_by_hand():
    x = np.zeros(32, np.float32)
    x[:8] = [6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25]      # every border, scale 1: ties to even
    codes, s = R.quantise_fp4(x, 1.0)
    assert list(codes[:8]) == [7, 6, 6, 4, 4, 2, 2, 0] and s[0] == 0x38 and s[1] == 0 and not codes[16:].any()
    tiles = R.pack_tiles(codes.reshape(1, 1, 1, 32).repeat(16, 1), s.reshape(1, 1, 1, 2).repeat(16, 1), True)
    assert tiles.shape == (1, 1, 9 * 32)
    assert np.array_equal(R.tile_values(tiles, True)[0, 3, 0, :8], [6, 4, 4, 2, 2, 1, 1, 0])


def test_reference_attention_by_hand():
    # one row, two keys, a window of one: the row is its own value
    k = np.zeros((1, 16, 1, 4)); v = np.arange(64.0).reshape(1, 16, 1, 4)
    q = np.ones((1, 1, 4))
    out, _, _, n = R.attention(q, k, v, np.zeros((1, 1), np.int32), [2], [1], 1.0, window=1)
    assert np.array_equal(out[0, 0], v[0, 1, 0]) and n[0, 0, 0] == 1
    out, _, _, _ = R.attention(q, k, v, np.zeros((1, 1), np.int32), [2], [1], 1.0, slopes=np.array([math.log(3.0)]))
    assert np.allclose(out[0, 0], 0.25 * v[0, 0, 0] + 0.75 * v[0, 1, 0])
    k[0, 0] = 100.0                                         # capped: scores 2 tanh(200), 0
    out, _, _, _ = R.attention(q, k, v, np.zeros((1, 1), np.int32), [2], [1], 1.0, softcap=2.0)
    p = math.exp(2) / (math.exp(2) + 1)
    assert np.allclose(out[0, 0], p * v[0, 0, 0] + (1 - p) * v[0, 1, 0])


def test_strided_4bit_write_refusals(lib):
    w = lib.pa_paged_kv_write_fp4_strided
    a = dict(key=F, ks=1024, value=F, vs=1024, kc=F, vc=F, slots=F, T=4, nb=8, hkv=8, d=128, bs=16, dt=0, a=1.0, b=1.0)
    for kw, status in ((dict(ks=1020), INVALID), (dict(vs=0), INVALID), (dict(ks=1028), UNSUPPORTED),
                       (dict(vs=2052), UNSUPPORTED), (dict(key=F + 8), INVALID), (dict(value=None), INVALID),
                       (dict(T=-1), INVALID), (dict(d=96, ks=768, vs=768), UNSUPPORTED), (dict(a=0.0), INVALID),
                       (dict(T=0), 0)):
        assert w(*dict(a, **kw).values(), None) == status
