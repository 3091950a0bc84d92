"""What the wrappers hand to the library, on the CPU with a stand-in library."""
import pytest
import torch

import paged_kv_attention_decode_gb300 as pa
from tests._stand_in import StandIn, Stream, dev


@pytest.fixture
def lib(monkeypatch):
    return StandIn(monkeypatch)


@pytest.mark.parametrize("shape,dtype,elem", [
    ((6, 16, 8, 128), torch.float16, 2),       # 16-bit, token-major
    ((6, 8, 16, 128), torch.uint8, 1),         # FP8, head-major: fewer, as many and more heads than tokens
    ((6, 16, 16, 128), torch.uint8, 1),
    ((6, 40, 16, 128), torch.float8_e4m3fn, 1),
    ((6, 1, 16, 128), torch.uint8, 1),
    ((6, 5, 9 * 128), torch.uint8, 1),         # 4-bit tiles
    ((6, 3, 9 * 64), torch.uint8, 1),
])
def test_copy_blocks_passes_the_bytes_of_a_block(lib, shape, dtype, elem):
    k, v = (dev(torch.zeros(shape, dtype=torch.uint8).to(dtype)) for _ in range(2))
    pa.copy_blocks(k, v, dev(torch.zeros(2, 2, dtype=torch.int32)))
    (name, args), = lib.calls
    assert name == "pa_copy_blocks" and args[3:5] == (2, 6) and args[7] == elem
    block = 16 * args[5] * args[6] * args[7]                 # as the header defines it
    assert block == k[0].numel() * k.element_size()


@pytest.mark.parametrize("shape,dtype", [
    ((6, 8, 16), torch.float16), ((6, 2, 8, 16, 128), torch.uint8), ((6, 8, 8, 128), torch.float16),
    ((6, 3, 4, 24), torch.uint8),
])
def test_copy_blocks_refuses_other_pools(lib, shape, dtype):
    k, v = (dev(torch.zeros(shape, dtype=torch.uint8).to(dtype)) for _ in range(2))
    with pytest.raises(pa.PagedAttnError):
        pa.copy_blocks(k, v, dev(torch.zeros(2, 2, dtype=torch.int32)))
    assert not lib.calls


# ---- calls on a stream that is not the current one -------------------------

NB, HKV, HQ, D, B, T = 8, 2, 4, 128, 3, 3
SIDE = 0x7000


def z(*shape, dtype=torch.float16):
    return dev(torch.zeros(shape, dtype=dtype))


def pools(kind):
    shape = {"16": (NB, 16, HKV, D), "fp8": (NB, HKV, 16, D), "fp4": (NB, HKV, 9 * D)}[kind]
    return tuple(z(*shape, dtype=torch.float16 if kind == "16" else torch.uint8) for _ in range(2))


def wrappers():
    """name -> call(**kw) of every wrapper that makes tensors of its own."""
    q, key = z(T, HQ, D), z(T, HKV, D)
    bt, sl = z(B, 4, dtype=torch.int32), dev(torch.full((B,), 20, dtype=torch.int32))
    cu = dev(torch.arange(B + 1, dtype=torch.int32))
    slots, pos, cs = z(T, dtype=torch.int64), z(T, dtype=torch.int64), z(30, D, dtype=torch.float32)
    p16, p8, p4 = pools("16"), pools("fp8"), pools("fp4")
    rope = (slots, pos, cs)
    return {
        "slot_mapping": lambda **kw: pa.slot_mapping(bt, sl, None, B, NB, **kw),
        "decode": lambda **kw: pa.paged_attention_decode(q, *p16, bt, sl, 0.1, **kw),
        "prefill": lambda **kw: pa.paged_attention_prefill(q, *p16, bt, sl, cu, 0.1, 1, 20, **kw),
        "decode_fp8": lambda **kw: pa.paged_attention_decode_fp8(q, *p8, bt, sl, 0.1, 1.0, 1.0, **kw),
        "prefill_fp8": lambda **kw: pa.paged_attention_prefill_fp8(q, *p8, bt, sl, cu, 0.1, 1.0, 1.0, 9, 20, **kw),
        "decode_fp4": lambda **kw: pa.paged_attention_decode_fp4(q, *p4, bt, sl, 0.1, 1.0, 1.0, **kw),
        "prefill_fp4": lambda **kw: pa.paged_attention_prefill_fp4(q, *p4, bt, sl, cu, 0.1, 1.0, 1.0, 9, 20, **kw),
        "decode_mod": lambda **kw: pa.paged_attention_decode_mod(q, *p16, bt, sl, 0.1, window=5, **kw),
        "prefill_mod": lambda **kw: pa.paged_attention_prefill_mod(q, *p16, bt, sl, cu, 0.1, 9, 20, window=5, **kw),
        "rope": lambda **kw: pa.paged_rope_kv_write(q, key, key, *p16, *rope, **kw),
        "rope_fp8": lambda **kw: pa.paged_rope_kv_write_fp8(q, key, key, *p8, *rope, 1.0, 1.0, **kw),
        "rope_fp4": lambda **kw: pa.paged_rope_kv_write_fp4(q, key, key, *p4, *rope, 1.0, 1.0, **kw),
        "unpack_fp4": lambda **kw: pa.paged_kv_unpack_fp4(*p4, 1.0, 1.0, torch.float16, **kw),
        "gather": lambda **kw: pa.paged_kv_gather(*p16, bt, sl, 20, **kw),
    }


NAMES = ["slot_mapping", "decode", "prefill", "decode_fp8", "prefill_fp8", "decode_fp4", "prefill_fp4", "decode_mod",
         "prefill_mod", "rope", "rope_fp8", "rope_fp4", "unpack_fp4", "gather"]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("as_handle", [False, True])
def test_a_given_stream_owns_what_the_call_makes(lib, name, as_handle):
    """Scratch belongs to the stream that the kernels run on: the allocator hands
    a freed block to the next tensor of the stream it was made on, at once."""
    call = wrappers()[name]
    lib.made.clear()
    out = call(stream=SIDE if as_handle else Stream(SIDE))
    assert lib.made and {s for _, _, s in lib.made} == {SIDE}
    (_, args), = lib.calls
    assert args[-1] == SIDE                                     # where the kernels run
    assert lib.now.cuda_stream == 0                             # the caller's stream is current again
    # the result may be used, and dropped, on the caller's stream
    for t in out if isinstance(out, tuple) else (out,):
        assert t.recorded == [0]


@pytest.mark.parametrize("name", NAMES)
def test_without_a_stream_the_current_one_serves(lib, name):
    call = wrappers()[name]
    for kw in ({}, {"stream": SIDE}):                           # (given, but the current one)
        lib.made.clear(), lib.calls.clear()
        lib.now = Stream(SIDE)
        out = call(**kw)
        assert {s for _, _, s in lib.made} == {SIDE} and lib.calls[0][1][-1] == SIDE
        for t in out if isinstance(out, tuple) else (out,):
            assert not hasattr(t, "recorded")


@pytest.mark.parametrize("handle", [0, 1])
def test_the_default_streams_handles(lib, handle):
    """0 and 1 both name the legacy default stream."""
    lib.now = Stream(SIDE)
    call = wrappers()["decode_mod"]
    lib.made.clear()
    call(stream=handle)
    assert {s for _, _, s in lib.made} == {0} and lib.calls[0][1][-1] == 0


@pytest.mark.parametrize("name", ["decode", "prefill_fp8", "prefill_fp4", "decode_mod"])
def test_given_outputs_and_workspaces_stay_the_callers(lib, name):
    call = wrappers()[name]
    out, ws = z(T, HQ, D), z(8192, dtype=torch.uint8)
    lib.made.clear()
    assert call(stream=Stream(SIDE), out=out, workspace=ws) is out
    assert not lib.made and not hasattr(out, "recorded") and not hasattr(ws, "recorded")
    assert ws.data_ptr() in lib.calls[0][1] and lib.calls[0][1][-1] == SIDE


def test_a_query_rotated_in_place_on_a_given_stream(lib):
    q, key = z(T, HQ, D), z(T, HKV, D)
    res = pa.paged_rope_kv_write(q, key, key, *pools("16"), z(T, dtype=torch.int64), z(T, dtype=torch.int64),
                                 z(30, D, dtype=torch.float32), q_out=q, stream=Stream(SIDE))
    assert res is q and not hasattr(q, "recorded") and lib.calls[0][1][-1] == SIDE


# ---- what a refusal names ---------------------------------------------------

def strided(t):
    """The same shape and values, not contiguous."""
    return dev(torch.stack([t.as_subclass(torch.Tensor)] * 2, -1)[..., 0])


class Elsewhere(type(dev(torch.zeros(1)))):
    """A tensor of another device than the current one."""

    def get_device(self):
        return 1


def elsewhere(t):
    return t.as_subclass(Elsewhere)


def args_of(call):
    q, key = z(T, HQ, D), z(T, HKV, D)
    kind = "fp4" if "fp4" in call else "fp8" if "fp8" in call else "16"
    k, v = pools(kind)
    tables = dict(block_tables=z(B, 4, dtype=torch.int32), seq_lens=z(B, dtype=torch.int32))
    scales = {} if kind == "16" else dict(k_scale=1.0, v_scale=1.0)
    if "rope" in call:
        return dict(q=q, key=key, value=z(T, HKV, D), k_cache=k, v_cache=v, slot_mapping=z(T, dtype=torch.int64),
                    positions=z(T, dtype=torch.int64), cos_sin=z(30, D, dtype=torch.float32), q_out=z(T, HQ, D),
                    **scales)
    if "kv_write" in call:
        return dict(key=key, value=z(T, HKV, D), k_cache=k, v_cache=v, slot_mapping=z(T, dtype=torch.int64), **scales)
    if "unpack" in call:
        return dict(k_cache=k, v_cache=v, dtype=torch.float16, **scales)
    a = dict(q=q, k_cache=k, v_cache=v, scale=0.1, max_seq_len=20, out=z(T, HQ, D),
             workspace=z(8192, dtype=torch.uint8), **tables, **scales)
    if "prefill" in call:
        a.update(cu_q_lens=z(B + 1, dtype=torch.int32), max_q_len=1)
    if "mod" in call:
        a.update(alibi_slopes=z(HQ, dtype=torch.float32))
    return a


CALLS = ["paged_rope_kv_write", "paged_rope_kv_write_fp8", "paged_rope_kv_write_fp4", "paged_kv_write_fp4",
         "paged_kv_unpack_fp4", "paged_attention_decode_fp4", "paged_attention_prefill_fp4",
         "paged_attention_decode_mod", "paged_attention_prefill_mod"]


def test_a_4bit_write_takes_slices_of_fused_rows(lib):
    """As the rotating writes do: the rows' stride goes to the library."""
    fused = z(T, (HQ + 2 * HKV) * D)
    k, v = (fused[:, (HQ + i * HKV) * D:(HQ + (i + 1) * HKV) * D].unflatten(1, (HKV, D)) for i in (0, 1))
    p = pools("fp4")
    for a, b, ks, vs in ((k, v, fused.shape[1], fused.shape[1]), (k, v.contiguous(), fused.shape[1], HKV * D),
                         (k[:1], v[:1], HKV * D, HKV * D)):
        lib.calls.clear()
        pa.paged_kv_write_fp4(a, b, *p, z(T, dtype=torch.int64), 1.0, 1.0)
        (_, args), = lib.calls
        assert args[:4] == (a.data_ptr(), ks, b.data_ptr(), vs)


@pytest.mark.parametrize("call", CALLS)
def test_good_arguments_are_taken(lib, call):
    getattr(pa, call)(**args_of(call))
    assert len(lib.calls) == 1


def as_type(dtype):
    return lambda t: dev(t.as_subclass(torch.Tensor).to(dtype))


def fewer(t):
    return dev(t.as_subclass(torch.Tensor)[:-1].clone())


ROPE, ATTN = CALLS[:3], CALLS[5:]
REFUSALS = [
    # calls, argument, what is wrong with it, words of the message
    (CALLS[:3] + CALLS[4:], "k_cache", elsewhere, "current CUDA device"),
    (CALLS, "v_cache", elsewhere, "current CUDA device"),
    (ROPE + CALLS[3:4], "slot_mapping", elsewhere, "current CUDA device"),
    (ATTN, "workspace", elsewhere, "current CUDA device"),
    (ROPE, "k_cache", strided, "k_cache and v_cache: contiguous"),
    (ROPE[:2], "v_cache", fewer, "k_cache and v_cache: contiguous, of one shape"),
    (CALLS[3:], "k_cache", strided, "contiguous"),
    (CALLS[3:4], "key", strided, "head rows"),
    (CALLS[3:4], "slot_mapping", strided, "contiguous"),
    (ATTN, "q", strided, "contiguous"),
    (ATTN, "workspace", strided, "contiguous"),
    (ATTN, "block_tables", strided, "contiguous"),
    (CALLS[7:], "alibi_slopes", strided, "contiguous"),
    (ROPE, "q", strided, "head rows"),
    (ROPE, "value", strided, "head rows"),
    (ROPE, "q_out", strided, "head rows"),
    (ROPE, "q_out", as_type(torch.bfloat16), "q_out: the shape and dtype of q"),
    (ROPE, "q_out", fewer, "q_out: the shape and dtype of q"),
    (ROPE, "q", fewer, "q/key/value shape"),
    (ROPE, "key", as_type(torch.bfloat16), "dtype"),
    (ROPE + CALLS[3:4], "slot_mapping", fewer, "slot_mapping: int64"),
    (ROPE + CALLS[3:4], "slot_mapping", as_type(torch.int32), "slot_mapping: int64"),
    (ROPE, "positions", fewer, "positions: int64"),
    (ROPE, "positions", strided, "positions: int64"),
    (ROPE, "cos_sin", as_type(torch.float64), "cos_sin: float32"),
    (ROPE, "cos_sin", strided, "cos_sin: float32"),
    (CALLS[3:4], "value", fewer, "key/value/cache shapes"),
    (ATTN, "seq_lens", as_type(torch.int64), "int32 tables"),
    (ATTN, "block_tables", fewer, "table shapes"),
    (ATTN, "out", fewer, "out shape/dtype"),
    (ATTN, "out", as_type(torch.float32), "out shape/dtype"),
    (CALLS[6:9:2], "cu_q_lens", fewer, "cu_q_lens"),
    (CALLS[7:], "alibi_slopes", fewer, "alibi_slopes: float32"),
    (CALLS[7:], "alibi_slopes", as_type(torch.float16), "alibi_slopes: float32"),
    (CALLS[7:], "v_cache", fewer, "cache shape/dtype"),
    (CALLS[5:7], "v_cache", fewer, "4-bit pools"),
    (CALLS[5:7], "k_cache", as_type(torch.float16), "4-bit pools"),
]


@pytest.mark.parametrize("call,arg,change,words", [(c, a, f, w) for cs, a, f, w in REFUSALS for c in cs])
def test_refusals_name_what_is_wrong(lib, call, arg, change, words):
    good = args_of(call)
    with pytest.raises(pa.PagedAttnError) as e:
        getattr(pa, call)(**dict(good, **{arg: change(good[arg])}))
    assert words in str(e.value) and not lib.calls


@pytest.mark.parametrize("call", ["paged_attention_decode_mod", "paged_attention_prefill_mod"])
@pytest.mark.parametrize("window,passed", [(0, 0), (7, 7), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31, 2 ** 31 - 1),
                                           (2 ** 32, 2 ** 31 - 1), (2 ** 32 + 5, 2 ** 31 - 1),
                                           (2 ** 63 - 1, 2 ** 31 - 1), (-3, -3), (-2 ** 32, -2 ** 31),
                                           (-2 ** 32 + 9, -2 ** 31)])
def test_a_window_past_32_bits_is_no_other_window(lib, call, window, passed):
    """(a C int would take its low bits: a window of 2^32 + 5 would be one of 5)"""
    import ctypes
    getattr(pa, call)(**dict(args_of(call), window=window))
    (name, args), = lib.calls
    at = 12 if "decode" in call else 15     # behind scale and softcap
    assert args[at - 2:at] == (0.1, 0.0) and ctypes.c_int(args[at]).value == passed


@pytest.mark.parametrize("change,words", [
    (dict(out=z(2, dtype=torch.int64)), "out: int64"), (dict(out=z(3, dtype=torch.int32)), "out: int64"),
    (dict(block_tables=z(2, 4, dtype=torch.int32)), "table shapes"),
    (dict(cu_q_lens=z(3, dtype=torch.int32)), "table shapes"), (dict(cu_q_lens=z(4, dtype=torch.int64)), "table shapes"),
])
def test_slot_mapping_refuses_short_arrays(lib, change, words):
    good = dict(block_tables=z(3, 4, dtype=torch.int32), seq_lens=z(3, dtype=torch.int32),
                cu_q_lens=z(4, dtype=torch.int32), num_tokens=3, num_blocks=8, out=z(3, dtype=torch.int64))
    pa.slot_mapping(**good)
    assert len(lib.calls) == 1
    with pytest.raises(pa.PagedAttnError, match=words):
        pa.slot_mapping(**dict(good, **change))
    assert len(lib.calls) == 1
