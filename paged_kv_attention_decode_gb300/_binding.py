"""ctypes binding of libpagedattn.so (declared in include/pagedattn.h).

Argument marshalling only: shape/dtype/device checks, ``data_ptr()`` and the
current CUDA stream go in, a status code comes out.  Every step of the path
runs in the library's kernels; there is no fallback of any kind.  Scratch
space is allocated here with torch (caller-owned memory for the library), on
the stream that the call runs on: torch's current one, or the `stream` given
(a torch stream or a handle; the caller orders it with the inputs' stream).
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "libpagedattn.so"

PA_BLOCK_SIZE = 16
PA_DEFAULT_PARTITION = 512
_DTYPES = {torch.float16: 0, torch.bfloat16: 1}
_STATUS = {0: "PA_OK", 1: "PA_ERR_INVALID_ARG", 2: "PA_ERR_UNSUPPORTED",
           3: "PA_ERR_WORKSPACE_TOO_SMALL", 4: "PA_ERR_CUDA"}

_p = ctypes.c_void_p
_i32 = ctypes.c_int
_f32 = ctypes.c_float
_i64 = ctypes.c_int64
_sz = ctypes.c_size_t

# q_out, q, key and value with their token strides, the pools, slots, positions,
# the cos/sin table and the sizes (the entry points differ after these)
_ROPE = [_p, _i64, _p, _i64, _p, _i64, _p, _i64, _p, _p, _p, _p, _p] + [_i32] * 9

_SIGNATURES = {
    "pa_version": (_i32, []),
    "pa_status_string": (ctypes.c_char_p, [_i32]),
    "pa_slot_mapping": (_i32, [_p, _p, _i32, _p, _p, _i32, _i32, _i32, _i32, _p]),
    "pa_paged_kv_write": (_i32, [_p, _p, _p, _p, _p, _i32, _i32, _i32, _i32, _i32, _i32, _p]),
    "pa_decode_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32, _i32]),
    "pa_paged_attention_decode": (_i32, [_p, _p, _p, _p, _p, _i32, _p, _i32, _i32, _i32, _f32,
                                         _i32, _i32, _i32, _i32, _i32, _p, _sz, _i32, _p]),
    "pa_prefill_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32, _i32]),
    "pa_paged_attention_prefill": (_i32, [_p, _p, _p, _p, _p, _i32, _p, _p, _i32, _i32, _i32,
                                          _i32, _i32, _f32, _i32, _i32, _i32, _i32, _p, _sz,
                                          _i32, _p]),
    "pa_get_device_error": (_i32, [ctypes.POINTER(_i32), _i32, _p]),
    "pa_paged_attention_decode_noalloc": (_i32, [_p, _p, _p, _p, _p, _i32, _p, _i32, _i32, _i32, _f32,
                                                 _i32, _i32, _i32, _i32, _i32, _i32, _p]),
    "pa_paged_kv_write_fp8": (_i32, [_p, _p, _p, _p, _p, _i32, _i32, _i32, _i32, _i32, _i32, _f32, _f32, _p]),
    "pa_paged_attention_decode_fp8": (_i32, [_p, _p, _p, _p, _p, _i32, _p, _i32, _i32, _i32, _f32, _f32, _f32,
                                             _i32, _i32, _i32, _i32, _i32, _p, _sz, _i32, _p]),
    "pa_prefill_fp8_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32, _i32, _i32, _i32, ctypes.c_int64]),
    "pa_paged_attention_prefill_fp8": (_i32, [_p, _p, _p, _p, _p, _i32, _p, _p, _i32, _i32, _i32, _i32, _i32,
                                              _f32, _f32, _f32, _i32, _i32, _i32, _i32, _p, _sz, _i32, _p]),
    "pa_paged_rope_kv_write": (_i32, _ROPE + [_i32, _p]),
    "pa_paged_rope_kv_write_fp8": (_i32, _ROPE + [_i32, _f32, _f32, _p]),
    "pa_paged_rope_kv_write_fp4": (_i32, _ROPE + [_i32, _f32, _f32, _p]),
    "pa_fp4_tile_bytes": (_i32, [_i32]),
    "pa_paged_kv_write_fp4": (_i32, [_p, _p, _p, _p, _p, _i32, _i32, _i32, _i32, _i32, _i32, _f32, _f32, _p]),
    "pa_paged_kv_write_fp4_strided": (_i32, [_p, _i64, _p, _i64, _p, _p, _p] + [_i32] * 6 + [_f32, _f32, _p]),
    "pa_paged_kv_unpack_fp4": (_i32, [_p, _p, _p, _p, _i32, _i32, _i32, _i32, _f32, _f32, _i32, _p]),
    "pa_paged_attention_decode_fp4": (_i32, [_p, _p, _p, _p, _p, _i32, _p, _i32, _i32, _i32, _f32, _f32, _f32,
                                             _i32, _i32, _i32, _i32, _i32, _p, _sz, _i32, _p]),
    "pa_paged_attention_prefill_fp4": (_i32, [_p, _p, _p, _p, _p, _i32, _p, _p, _i32, _i32, _i32, _i32, _i32,
                                              _f32, _f32, _f32, _i32, _i32, _i32, _i32, _p, _sz, _i32, _p]),
    "pa_prefill_mod_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32, _i32, _i32]),
    "pa_prefill_fp4_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32, _i32, _i32, _i32, ctypes.c_int64]),
    "pa_paged_attention_decode_mod": (_i32, [_p, _p, _p, _p, _p, _i32, _p, _i32, _i32, _i32, _f32, _f32, _i32, _p,
                                             _i32, _i32, _i32, _i32, _i32, _p, _sz, _i32, _p]),
    "pa_paged_attention_prefill_mod": (_i32, [_p, _p, _p, _p, _p, _i32, _p, _p, _i32, _i32, _i32, _i32, _i32,
                                              _f32, _f32, _i32, _p, _i32, _i32, _i32, _i32, _p, _sz, _i32, _p]),
    "pa_cross_workspace_bytes": (_sz, [_i32, _i32, _i32]),
    "pa_paged_cross_attention": (_i32, [_p, _p, _p, _p, _p, _i32, _p, _p, _i32, _i32, _i32, _i32, _i32, _f32,
                                        _i32, _i32, _i32, _i32, _p, _sz, _i32, _p]),
    "pa_beam_select_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32, _i32]),
    "pa_beam_select": (_i32, [_p, _p, _p, _p, _p, _i64, _p, _p, _i32, _i32, _i32, _i32, _i32, _i32, _p, _sz, _p]),
    "pa_beam_reorder": (_i32, [_p, _p, _i32, _p, _p, _i32, _i32, _p, _p, _i32, _i32, _i32, _i32, _i32, _i32, _p]),
    "pa_copy_blocks": (_i32, [_p, _p, _p, _i32, _i32, _i32, _i32, _i32, _p]),
    "pa_decode_partition": (_i32, [_i32, _i32]),
    "pa_decode_partition_for": (_i32, [_i32, _i32, _i32, _i32]),
    "pa_selftest_wait_timeout": (_i32, [_p]),
    "pa_paged_kv_gather": (_i32, [_p, _p, _p, _p, _p, _i32, _p, _p, _i32, _i32, _i32, _i32, _i32, _i32, _p]),
}


class PagedAttnError(RuntimeError):
    """A libpagedattn call returned a nonzero status, or the library is missing."""


_lib = None


def library_path() -> str:
    return os.path.join(_HERE, _LIB_NAME)


def load_library():
    """Load libpagedattn.so from the package directory (raises if it is not built)."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise PagedAttnError(
            f"{path} is missing: build it first (python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _check(rc: int, what: str) -> None:
    if rc != 0:
        raise PagedAttnError(f"{what} failed: {_STATUS.get(rc, rc)}")


def _stream(stream) -> int:
    if stream is None:   # the current stream's handle, without a Stream object around it
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _dt(t: torch.Tensor) -> int:
    if t.dtype not in _DTYPES:
        raise PagedAttnError(f"unsupported dtype {t.dtype}")
    return _DTYPES[t.dtype]


def _need(cond: bool, msg: str) -> None:
    if not cond:
        raise PagedAttnError(msg)


def _cuda(*ts):
    for t in ts:
        if t is not None:
            _need(t.is_cuda and t.is_contiguous(), "tensors must be contiguous CUDA tensors")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _given(stream, call, *args, **kw):
    """`call(*args, **kw)` with the given stream as torch's current one.

    The calls make scratch that is dropped as they return, while their kernels
    still run; the allocator hands it to the next tensor of the stream it was
    made on, at once, so that must be the kernels' stream.  What is read on the
    way (lengths on the host, sums) is ordered with that stream's work too.  A
    tensor that the call made and returns may be used and dropped on the stream
    that was current."""
    before = torch.cuda.current_stream()
    handle = _stream(stream)
    if handle == before.cuda_stream:
        return call(*args, **kw)
    if not isinstance(stream, torch.cuda.Stream):   # 0 and 1: the legacy default stream
        stream = torch.cuda.ExternalStream(handle) if handle > 1 else torch.cuda.default_stream()
    with torch.cuda.stream(stream):
        made = call(*args, **kw)
    theirs = [*args, *kw.values()]
    theirs += [t for a in theirs if isinstance(a, (tuple, list)) for t in a]
    for t in made if isinstance(made, tuple) else (made,):
        if not any(t is x for x in theirs):
            t.record_stream(before)
    return made


# --------------------------------------------------------------------------

def slot_mapping(block_tables: torch.Tensor, seq_lens: torch.Tensor, cu_q_lens, num_tokens: int,
                 num_blocks: int, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """int64 slot of every new token (the last q_len positions of each sequence);
    -1 for rows behind the last sequence's."""
    if stream is not None:
        return _given(stream, slot_mapping, block_tables, seq_lens, cu_q_lens, num_tokens, num_blocks, out)
    _cuda(block_tables, seq_lens, cu_q_lens)
    _need(block_tables.dtype == torch.int32 and seq_lens.dtype == torch.int32, "int32 tables")
    B = seq_lens.shape[0]
    if out is None:
        out = torch.empty(num_tokens, dtype=torch.int64, device=seq_lens.device)
        if B == 0:   # (the library returns at once)
            out.fill_(-1)
    _cuda(out)
    _need(out.dtype == torch.int64 and out.numel() >= num_tokens, "out: int64 [num_tokens]")
    _need(block_tables.dim() == 2 and block_tables.shape[0] >= B
          and (cu_q_lens is None or (cu_q_lens.dtype == torch.int32 and cu_q_lens.numel() == B + 1)), "table shapes")
    rc = load_library().pa_slot_mapping(out.data_ptr(), block_tables.data_ptr(), block_tables.shape[1],
                                        seq_lens.data_ptr(), _ptr(cu_q_lens), B, num_tokens,
                                        num_blocks, PA_BLOCK_SIZE, _stream(None))
    _check(rc, "pa_slot_mapping")
    return out


def paged_kv_write(key: torch.Tensor, value: torch.Tensor, k_cache: torch.Tensor,
                   v_cache: torch.Tensor, slot_mapping: torch.Tensor, stream=None) -> None:
    """In place: k_cache/v_cache[slot // 16, slot % 16] = key/value rows (slot < 0: skipped)."""
    _cuda(key, value, k_cache, v_cache, slot_mapping)
    _need(slot_mapping.dtype == torch.int64, "slot_mapping must be int64")
    NB, bs, H, D = k_cache.shape
    T = key.shape[0]
    _need(tuple(key.shape) == (T, H, D) and value.shape == key.shape, "key/value shape")
    _need(v_cache.shape == k_cache.shape and k_cache.dtype == key.dtype == value.dtype == v_cache.dtype,
          "cache shape/dtype")
    _need(slot_mapping.numel() >= T, "slot_mapping too short")
    rc = load_library().pa_paged_kv_write(key.data_ptr(), value.data_ptr(), k_cache.data_ptr(),
                                          v_cache.data_ptr(), slot_mapping.data_ptr(), T, NB, H, D,
                                          bs, _dt(key), _stream(stream))
    _check(rc, "pa_paged_kv_write")


def selftest_wait_timeout(stream=None) -> None:
    """Enqueue the failure-path self-test (a bounded wait that runs out after
    about a second and records PA_DEVERR_TIMEOUT)."""
    _check(load_library().pa_selftest_wait_timeout(_stream(stream)), "pa_selftest_wait_timeout")


def decode_partition(max_seq_len: int, partition_size: int = 0) -> int:
    """Partition length (tokens) a decode call uses; 0 selects the automatic one."""
    n = int(load_library().pa_decode_partition(max_seq_len, partition_size))
    _need(n > 0, "invalid max_seq_len or partition_size")
    return n


def decode_partition_for(num_seqs: int, num_q_heads: int, num_kv_heads: int, max_seq_len: int) -> int:
    """Partition length that gives a decode call of these sizes enough work
    items for the GPU (at most that of `decode_partition(max_seq_len)`)."""
    n = int(load_library().pa_decode_partition_for(num_seqs, num_q_heads, num_kv_heads, max_seq_len))
    _need(n > 0, "invalid sizes")
    return n


def decode_workspace_bytes(num_seqs: int, num_q_heads: int, head_dim: int, max_seq_len: int,
                           partition_size: int = 0) -> int:
    return int(load_library().pa_decode_workspace_bytes(num_seqs, num_q_heads, head_dim, max_seq_len,
                                                        partition_size))


def prefill_workspace_bytes(num_seqs: int, num_tokens: int, num_q_heads: int, head_dim: int,
                            max_seq_len: int) -> int:
    return int(load_library().pa_prefill_workspace_bytes(num_seqs, num_tokens, num_q_heads, head_dim,
                                                         max_seq_len))


def prefill_fp8_workspace_bytes(num_seqs: int, num_tokens: int, num_q_heads: int, num_kv_heads: int,
                                head_dim: int, max_seq_len: int, max_blocks_per_seq: int,
                                chunk_kv_tokens: int) -> int:
    return int(load_library().pa_prefill_fp8_workspace_bytes(num_seqs, num_tokens, num_q_heads, num_kv_heads,
                                                             head_dim, max_seq_len, max_blocks_per_seq,
                                                             chunk_kv_tokens))


def prefill_fp4_workspace_bytes(num_seqs: int, num_tokens: int, num_q_heads: int, num_kv_heads: int,
                                head_dim: int, max_seq_len: int, max_blocks_per_seq: int,
                                chunk_kv_tokens: int) -> int:
    return int(load_library().pa_prefill_fp4_workspace_bytes(num_seqs, num_tokens, num_q_heads, num_kv_heads,
                                                             head_dim, max_seq_len, max_blocks_per_seq,
                                                             chunk_kv_tokens))


def prefill_mod_workspace_bytes(num_seqs: int, num_tokens: int, num_q_heads: int, num_kv_heads: int,
                                head_dim: int, max_seq_len: int) -> int:
    return int(load_library().pa_prefill_mod_workspace_bytes(num_seqs, num_tokens, num_q_heads, num_kv_heads,
                                                             head_dim, max_seq_len))


def count_chunk_kv_tokens(seq_lens: torch.Tensor, cu_q_lens: torch.Tensor) -> int:
    """Sum of seq_lens over the rows with more than 8 new tokens (the FP8
    prefill copy's size argument), from host copies of the two arrays."""
    sl = seq_lens.detach().to("cpu", torch.int64)
    cu = cu_q_lens.detach().to("cpu", torch.int64)
    return int(sl[(cu[1:] - cu[:-1]) > 8].sum())


def _workspace(nbytes: int, device, workspace):
    if nbytes == 0:
        return workspace
    if workspace is not None and workspace.numel() * workspace.element_size() >= nbytes:
        return workspace
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def paged_attention_decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                           block_tables: torch.Tensor, seq_lens: torch.Tensor, scale: float,
                           max_seq_len: int | None = None, out: torch.Tensor | None = None,
                           partition_size: int = 0, workspace: torch.Tensor | None = None,
                           stream=None) -> torch.Tensor:
    """Decode attention: q [B, Hq, D] -> out [B, Hq, D] over the paged cache."""
    if stream is not None:
        return _given(stream, paged_attention_decode, q, k_cache, v_cache, block_tables, seq_lens, scale,
                      max_seq_len, out, partition_size, workspace)
    _cuda(q, k_cache, v_cache, block_tables, seq_lens, out, workspace)
    B, Hq, D = q.shape
    NB, bs, Hkv, D2 = k_cache.shape
    _need(D2 == D and v_cache.shape == k_cache.shape, "cache shape")
    _need(block_tables.dtype == torch.int32 and seq_lens.dtype == torch.int32, "int32 tables")
    if max_seq_len is None:
        max_seq_len = int(seq_lens.max().item()) if B else 0
    if out is None:
        out = torch.empty_like(q)
    nbytes = decode_workspace_bytes(B, Hq, D, max_seq_len, partition_size)
    workspace = _workspace(nbytes, q.device, workspace)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load_library().pa_paged_attention_decode(
        out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(),
        block_tables.shape[1], seq_lens.data_ptr(), B, max_seq_len, NB, float(scale), Hq, Hkv, D, bs,
        partition_size, _ptr(workspace), ws_bytes, _dt(q), _stream(None))
    _check(rc, "pa_paged_attention_decode")
    return out


def paged_attention_prefill(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                            block_tables: torch.Tensor, seq_lens: torch.Tensor,
                            cu_q_lens: torch.Tensor, scale: float, max_q_len: int,
                            max_seq_len: int, out: torch.Tensor | None = None,
                            workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Causal varlen attention of new query rows over the paged cache.

    Chunks of at most PA_VERIFY_MAX_Q (8) queries -- decodes and speculative
    verify steps -- run in the decode kernel, longer chunks in the prefill
    kernels."""
    if stream is not None:
        return _given(stream, paged_attention_prefill, q, k_cache, v_cache, block_tables, seq_lens, cu_q_lens,
                      scale, max_q_len, max_seq_len, out, workspace)
    _cuda(q, k_cache, v_cache, block_tables, seq_lens, cu_q_lens, out, workspace)
    T, Hq, D = q.shape
    NB, bs, Hkv, D2 = k_cache.shape
    _need(D2 == D and v_cache.shape == k_cache.shape, "cache shape")
    B = seq_lens.shape[0]
    _need(cu_q_lens.shape[0] == B + 1 and cu_q_lens.dtype == torch.int32, "cu_q_lens")
    if out is None:
        out = torch.empty_like(q)
    nbytes = prefill_workspace_bytes(B, T, Hq, D, max_seq_len)
    workspace = _workspace(nbytes, q.device, workspace)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load_library().pa_paged_attention_prefill(
        out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(),
        block_tables.shape[1], seq_lens.data_ptr(), cu_q_lens.data_ptr(), B, T, max_q_len, max_seq_len,
        NB, float(scale), Hq, Hkv, D, bs, _ptr(workspace), ws_bytes, _dt(q), _stream(None))
    _check(rc, "pa_paged_attention_prefill")
    return out


def copy_blocks(k_cache: torch.Tensor, v_cache: torch.Tensor, pairs: torch.Tensor, stream=None) -> None:
    """In place: block pairs[i, 1] of both pools receives block pairs[i, 0]
    (the copy-on-write step; pairs is a device int32 [n, 2] tensor).  Pools of
    any kind: 16-bit [NB, 16, Hkv, D], FP8 [NB, Hkv, 16, D], or 4-bit tiles
    [NB, Hkv, bytes]."""
    _cuda(k_cache, v_cache, pairs)
    _need(pairs.dtype == torch.int32 and pairs.dim() == 2 and pairs.shape[1] == 2, "pairs: int32 [n, 2]")
    _need(v_cache.shape == k_cache.shape and v_cache.dtype == k_cache.dtype, "cache shape/dtype")
    shape, elem = k_cache.shape, k_cache.element_size()
    NB = shape[0]
    if k_cache.dim() == 3:   # 4-bit tiles: 16 rows of codes and scales
        _need(elem == 1 and shape[2] % 16 == 0, "4-bit pools: bytes [NB, Hkv, fp4_tile_bytes]")
        H, D = shape[1], shape[2] // 16
    else:                    # 16 token rows, before the heads or (one-byte pools) after them
        _need(k_cache.dim() == 4 and (shape[1] == PA_BLOCK_SIZE or (elem == 1 and shape[2] == PA_BLOCK_SIZE)),
              "pools: [NB, 16, Hkv, D], or one-byte [NB, Hkv, 16, D]")
        H, D = shape[1] * shape[2] // PA_BLOCK_SIZE, shape[3]
    rc = load_library().pa_copy_blocks(k_cache.data_ptr(), v_cache.data_ptr(), pairs.data_ptr(), pairs.shape[0],
                                       NB, H, D, elem, _stream(stream))
    _check(rc, "pa_copy_blocks")


def paged_kv_gather(k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
                    seq_lens: torch.Tensor, max_seq_len: int, stream=None):
    """Test support: every sequence's live K/V rows, gathered through its block
    table into contiguous [sum(seq_lens), Hkv, D] tensors.  16-bit pools are
    [NB, 16, Hkv, D]; one-byte (FP8) pools are head-major [NB, Hkv, 16, D]."""
    if stream is not None:
        return _given(stream, paged_kv_gather, k_cache, v_cache, block_tables, seq_lens, max_seq_len)
    _cuda(k_cache, v_cache, block_tables, seq_lens)
    _need(block_tables.dtype == torch.int32 and seq_lens.dtype == torch.int32, "int32 tables")
    _need(v_cache.shape == k_cache.shape and v_cache.dtype == k_cache.dtype, "cache shape/dtype")
    if k_cache.element_size() == 1:
        NB, H, bs, D = k_cache.shape
    else:
        NB, bs, H, D = k_cache.shape
    B = seq_lens.shape[0]
    cu = torch.zeros(B + 1, dtype=torch.int32, device=seq_lens.device)
    torch.cumsum(seq_lens, 0, out=cu[1:])
    total = int(cu[-1])
    k_out = torch.empty(total, H, D, dtype=k_cache.dtype, device=k_cache.device)
    v_out = torch.empty_like(k_out)
    rc = load_library().pa_paged_kv_gather(k_out.data_ptr(), v_out.data_ptr(), k_cache.data_ptr(),
                                           v_cache.data_ptr(), block_tables.data_ptr(), block_tables.shape[1],
                                           seq_lens.data_ptr(), cu.data_ptr(), B, max_seq_len, NB, H, D,
                                           k_cache.element_size(), _stream(None))
    _check(rc, "pa_paged_kv_gather")
    return k_out, v_out


def device_error(clear: bool = True, stream=None) -> int:
    """Device error word (PA_DEVERR_* bits); synchronises the stream."""
    code = ctypes.c_int(0)
    _check(load_library().pa_get_device_error(ctypes.byref(code), int(clear), _stream(stream)),
           "pa_get_device_error")
    return code.value


# --------------------------------------------------------------------------
# FP8 (E4M3) cache
# --------------------------------------------------------------------------

def _u8(t: torch.Tensor) -> torch.Tensor:
    _need(t.element_size() == 1, "FP8 caches hold one byte per element")
    return t


def paged_kv_write_fp8(key: torch.Tensor, value: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                       slot_mapping: torch.Tensor, k_scale: float, v_scale: float, stream=None) -> None:
    """In place: E4M3 codes of key/value * (1 / scale) into the head-major FP8
    pools [NB, Hkv, 16, D] (slot < 0: skipped)."""
    _cuda(key, value, k_cache, v_cache, slot_mapping)
    _u8(k_cache), _u8(v_cache)
    _need(slot_mapping.dtype == torch.int64, "slot_mapping must be int64")
    NB, H, bs, D = k_cache.shape
    T = key.shape[0]
    _need(tuple(key.shape) == (T, H, D) and value.shape == key.shape and v_cache.shape == k_cache.shape,
          "key/value/cache shapes")
    rc = load_library().pa_paged_kv_write_fp8(key.data_ptr(), value.data_ptr(), k_cache.data_ptr(),
                                              v_cache.data_ptr(), slot_mapping.data_ptr(), T, NB, H, D, bs,
                                              _dt(key), float(k_scale), float(v_scale), _stream(stream))
    _check(rc, "pa_paged_kv_write_fp8")


def paged_attention_decode_fp8(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                               block_tables: torch.Tensor, seq_lens: torch.Tensor, scale: float, k_scale: float,
                               v_scale: float, max_seq_len: int | None = None, out: torch.Tensor | None = None,
                               partition_size: int = 0, workspace: torch.Tensor | None = None,
                               stream=None) -> torch.Tensor:
    """Decode attention over head-major FP8 (E4M3) pools [NB, Hkv, 16, 128]:
    q [B, Hq, 128] -> out [B, Hq, 128]."""
    if stream is not None:
        return _given(stream, paged_attention_decode_fp8, q, k_cache, v_cache, block_tables, seq_lens, scale,
                      k_scale, v_scale, max_seq_len, out, partition_size, workspace)
    _cuda(q, k_cache, v_cache, block_tables, seq_lens, out, workspace)
    _u8(k_cache), _u8(v_cache)
    B, Hq, D = q.shape
    NB, Hkv, bs, D2 = k_cache.shape
    _need(D2 == D and v_cache.shape == k_cache.shape, "cache shape")
    if max_seq_len is None:
        max_seq_len = int(seq_lens.max().item()) if B else 0
    if out is None:
        out = torch.empty_like(q)
    nbytes = decode_workspace_bytes(B, Hq, D, max_seq_len, partition_size)
    workspace = _workspace(nbytes, q.device, workspace)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load_library().pa_paged_attention_decode_fp8(
        out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(),
        block_tables.shape[1], seq_lens.data_ptr(), B, max_seq_len, NB, float(scale), float(k_scale),
        float(v_scale), Hq, Hkv, D, bs, partition_size, _ptr(workspace), ws_bytes, _dt(q), _stream(None))
    _check(rc, "pa_paged_attention_decode_fp8")
    return out


def paged_attention_prefill_fp8(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                block_tables: torch.Tensor, seq_lens: torch.Tensor, cu_q_lens: torch.Tensor,
                                scale: float, k_scale: float, v_scale: float, max_q_len: int, max_seq_len: int,
                                out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                                stream=None, chunk_kv_tokens: int | None = None) -> torch.Tensor:
    """Causal varlen attention of new query rows over head-major FP8 (E4M3)
    pools [NB, Hkv, 16, 128] (decodes, speculative-verify rows and prefill
    chunks in one call).  `chunk_kv_tokens` sizes the chunks' 16-bit copy
    (see `count_chunk_kv_tokens()`); when it is None and a chunk can be longer than
    8 queries, it is computed from host copies of seq_lens and cu_q_lens."""
    if stream is not None:
        return _given(stream, paged_attention_prefill_fp8, q, k_cache, v_cache, block_tables, seq_lens, cu_q_lens,
                      scale, k_scale, v_scale, max_q_len, max_seq_len, out, workspace,
                      chunk_kv_tokens=chunk_kv_tokens)
    _cuda(q, k_cache, v_cache, block_tables, seq_lens, cu_q_lens, out, workspace)
    _u8(k_cache), _u8(v_cache)
    T, Hq, D = q.shape
    NB, Hkv, bs, D2 = k_cache.shape
    _need(D2 == D and v_cache.shape == k_cache.shape, "cache shape")
    B = seq_lens.shape[0]
    _need(cu_q_lens.shape[0] == B + 1 and cu_q_lens.dtype == torch.int32, "cu_q_lens")
    if out is None:
        out = torch.empty_like(q)
    if max_q_len > 8 and B > 0 and T > 0:
        if chunk_kv_tokens is None:
            chunk_kv_tokens = count_chunk_kv_tokens(seq_lens, cu_q_lens)
        nbytes = prefill_fp8_workspace_bytes(B, T, Hq, Hkv, D, max_seq_len, block_tables.shape[1],
                                             chunk_kv_tokens)
    else:
        nbytes = prefill_workspace_bytes(B, T, Hq, D, max_seq_len)
    workspace = _workspace(nbytes, q.device, workspace)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load_library().pa_paged_attention_prefill_fp8(
        out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(),
        block_tables.shape[1], seq_lens.data_ptr(), cu_q_lens.data_ptr(), B, T, max_q_len, max_seq_len, NB,
        float(scale), float(k_scale), float(v_scale), Hq, Hkv, D, bs, _ptr(workspace), ws_bytes, _dt(q),
        _stream(None))
    _check(rc, "pa_paged_attention_prefill_fp8")
    return out


# --------------------------------------------------------------------------
# Rotation and append; 4-bit (E2M1) cache
# --------------------------------------------------------------------------

# These calls check their arguments with one condition on the way (a serving
# step makes thousands of them) and find out what was wrong only when it fails.
_cuda_device = getattr(torch._C, "_cuda_getDevice", None)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_F16, _BF16, _F32, _I32T, _I64T = torch.float16, torch.bfloat16, torch.float32, torch.int32, torch.int64


def _refuse(name: str, *checks) -> None:
    """Raise for the first (condition, message) that does not hold."""
    for ok, msg in checks:
        _need(ok, msg)
    _need(False, f"{name}: invalid arguments")


def _current(dev: int, *ts) -> bool:
    """Every tensor on CUDA device `dev`, and that one current."""
    return dev >= 0 and all(t is None or t.get_device() == dev for t in ts) and torch.cuda.current_device() == dev


def _rope(name, q, key, value, k_cache, v_cache, slot_mapping, positions, cos_sin, interleaved, q_out, pool, scales):
    """The three rotate-and-append calls; `pool` is (num_blocks, num_kv_heads, head_dim, block_size)."""
    NB, H, D, bs = pool
    shape = key.shape
    T, H2, D2 = shape
    qshape = q.shape
    T2, Hq, D3 = qshape
    dtype = q.dtype
    dev = q.get_device()
    qs, qh, q1 = q.stride()
    ks, kh, k1 = key.stride()
    vs, vh, v1 = value.stride()
    if q_out is None:
        q_out = torch.empty_like(q) if q.is_contiguous() else torch.empty(qshape, dtype=dtype, device=q.device)
        os = Hq * D
        out_ok = True
    else:
        os, oh, o1 = q_out.stride()
        out_ok = (q_out.shape == qshape and q_out.dtype == dtype and q_out.get_device() == dev and o1 == 1
                  and (oh == D or Hq <= 1))
    if T <= 1:   # the stride of a single row says nothing
        qs = os = Hq * D
        ks = vs = H * D
    if not (dev >= 0 and _cuda_device() == dev and key.get_device() == dev and value.get_device() == dev
            and k_cache.get_device() == dev and v_cache.get_device() == dev and slot_mapping.get_device() == dev
            and positions.get_device() == dev and cos_sin.get_device() == dev
            and T2 == T and H2 == H and D2 == D and D3 == D and value.shape == shape and out_ok
            and key.dtype == dtype and value.dtype == dtype and (dtype == _F16 or dtype == _BF16)
            and q1 == 1 and k1 == 1 and v1 == 1 and (qh == D or Hq <= 1) and ((kh == D and vh == D) or H <= 1)
            and v_cache.shape == k_cache.shape and k_cache.is_contiguous() and v_cache.is_contiguous()
            and slot_mapping.dtype == _I64T and slot_mapping.is_contiguous() and slot_mapping.numel() >= T
            and positions.dtype == _I64T and positions.is_contiguous() and positions.numel() >= T
            and cos_sin.dtype == _F32 and cos_sin.dim() == 2 and cos_sin.is_contiguous()):
        _refuse(name,
                (_current(dev, key, value, k_cache, v_cache, slot_mapping, positions, cos_sin, q_out),
                 "tensors must be on the current CUDA device"),
                (T2 == T and H2 == H and D2 == D and D3 == D and value.shape == shape, "q/key/value shape"),
                (key.dtype == dtype and value.dtype == dtype, "q/key/value dtype"),
                (dtype in _DTYPES, f"unsupported dtype {dtype}"),
                (v_cache.shape == k_cache.shape and k_cache.is_contiguous() and v_cache.is_contiguous(),
                 "k_cache and v_cache: contiguous, of one shape"),
                (slot_mapping.dtype == _I64T and slot_mapping.is_contiguous() and slot_mapping.numel() >= T,
                 "slot_mapping: int64 [num_tokens]"),
                (positions.dtype == _I64T and positions.is_contiguous() and positions.numel() >= T,
                 "positions: int64 [num_tokens]"),
                (cos_sin.dtype == _F32 and cos_sin.dim() == 2 and cos_sin.is_contiguous(),
                 "cos_sin: float32 [max_positions, rot_dim]"),
                (q_out.shape == qshape and q_out.dtype == dtype, "q_out: the shape and dtype of q"),
                (False, "q, key, value and q_out: head rows must be dense within a token"))
    maxp, rot = cos_sin.shape
    rc = getattr(_lib or load_library(), name)(
        q_out.data_ptr(), os, q.data_ptr(), qs, key.data_ptr(), ks, value.data_ptr(), vs, k_cache.data_ptr(),
        v_cache.data_ptr(), slot_mapping.data_ptr(), positions.data_ptr(), cos_sin.data_ptr(), maxp, T, NB, Hq, H, D,
        rot, 1 if interleaved else 0, bs, 0 if dtype == _F16 else 1, *scales,
        _raw_stream(dev))
    if rc:
        _check(rc, name)
    return q_out


def paged_rope_kv_write(q: torch.Tensor, key: torch.Tensor, value: torch.Tensor, k_cache: torch.Tensor,
                        v_cache: torch.Tensor, slot_mapping: torch.Tensor, positions: torch.Tensor,
                        cos_sin: torch.Tensor, interleaved: bool = False, q_out: torch.Tensor | None = None,
                        stream=None) -> torch.Tensor:
    """Rotate the step's queries and keys by their positions and write keys and
    values into their slots of a 16-bit cache, in one pass; returns the rotated
    queries (`q_out`, which may be `q` itself).

    q [T, Hq, D], key/value [T, Hkv, D] may be slices of fused projection rows
    (any token stride that is a multiple of 8 elements).  cos_sin is float32
    [max_positions, rot_dim], cosines then sines; pairs are (i, i + rot_dim/2),
    or (2i, 2i + 1) when interleaved."""
    if stream is not None:
        return _given(stream, paged_rope_kv_write, q, key, value, k_cache, v_cache, slot_mapping, positions,
                      cos_sin, interleaved, q_out)
    NB, bs, H, D = k_cache.shape
    dtype = key.dtype
    if k_cache.dtype != dtype or v_cache.dtype != dtype:
        _need(False, "cache dtype")
    return _rope("pa_paged_rope_kv_write", q, key, value, k_cache, v_cache, slot_mapping, positions, cos_sin,
                 interleaved, q_out, (NB, H, D, bs), ())


def paged_rope_kv_write_fp8(q: torch.Tensor, key: torch.Tensor, value: torch.Tensor, k_cache: torch.Tensor,
                            v_cache: torch.Tensor, slot_mapping: torch.Tensor, positions: torch.Tensor,
                            cos_sin: torch.Tensor, k_scale: float, v_scale: float, interleaved: bool = False,
                            q_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """`paged_rope_kv_write` into head-major FP8 (E4M3) pools [NB, Hkv, 16, 128]."""
    if stream is not None:
        return _given(stream, paged_rope_kv_write_fp8, q, key, value, k_cache, v_cache, slot_mapping, positions,
                      cos_sin, k_scale, v_scale, interleaved, q_out)
    _u8(k_cache), _u8(v_cache)
    NB, H, bs, D = k_cache.shape
    return _rope("pa_paged_rope_kv_write_fp8", q, key, value, k_cache, v_cache, slot_mapping, positions, cos_sin,
                 interleaved, q_out, (NB, H, D, bs), (float(k_scale), float(v_scale)))


def fp4_tile_bytes(head_dim: int) -> int:
    """Bytes of one (block, kv head) tile of a 4-bit cache; its pools are uint8
    [num_blocks, num_kv_heads, fp4_tile_bytes(head_dim)]."""
    n = int(load_library().pa_fp4_tile_bytes(head_dim))
    _need(n > 0, "4-bit caches hold head_dim 64 or 128")
    return n


def _fp4_pool(k_cache: torch.Tensor, v_cache: torch.Tensor, D: int):
    """(num_blocks, num_kv_heads) of a pair of 4-bit pools of head_dim D."""
    shape = k_cache.shape
    if not (len(shape) == 3 and shape[2] == 9 * D and (D == 128 or D == 64) and v_cache.shape == shape
            and k_cache.element_size() == 1 and v_cache.element_size() == 1):
        _need(D == 128 or D == 64, "4-bit caches hold head_dim 64 or 128")
        _need(False, "4-bit pools: bytes [NB, Hkv, fp4_tile_bytes(head_dim)]")
    return shape[0], shape[1]


def paged_rope_kv_write_fp4(q: torch.Tensor, key: torch.Tensor, value: torch.Tensor, k_cache: torch.Tensor,
                            v_cache: torch.Tensor, slot_mapping: torch.Tensor, positions: torch.Tensor,
                            cos_sin: torch.Tensor, k_scale: float, v_scale: float, interleaved: bool = False,
                            q_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """`paged_rope_kv_write` into 4-bit pools [NB, Hkv, fp4_tile_bytes(D)]."""
    if stream is not None:
        return _given(stream, paged_rope_kv_write_fp4, q, key, value, k_cache, v_cache, slot_mapping, positions,
                      cos_sin, k_scale, v_scale, interleaved, q_out)
    D = key.shape[2]
    NB, H = _fp4_pool(k_cache, v_cache, D)
    return _rope("pa_paged_rope_kv_write_fp4", q, key, value, k_cache, v_cache, slot_mapping, positions, cos_sin,
                 interleaved, q_out, (NB, H, D, PA_BLOCK_SIZE), (float(k_scale), float(v_scale)))


def paged_kv_write_fp4(key: torch.Tensor, value: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                       slot_mapping: torch.Tensor, k_scale: float, v_scale: float, stream=None) -> None:
    """In place: E2M1 codes and E4M3 group scales of key/value into the 4-bit
    pools [NB, Hkv, fp4_tile_bytes(D)] (slot < 0: skipped).  key/value
    [T, Hkv, D] may be slices of fused projection rows, as in
    `paged_rope_kv_write`."""
    shape = key.shape
    T, H, D = shape
    NB, H2 = _fp4_pool(k_cache, v_cache, D)
    dtype = key.dtype
    dev = key.get_device()
    if not (dev >= 0 and _cuda_device() == dev and value.get_device() == dev and k_cache.get_device() == dev
            and v_cache.get_device() == dev and slot_mapping.get_device() == dev and H == H2
            and value.shape == shape and value.dtype == dtype and (dtype == _F16 or dtype == _BF16)
            and slot_mapping.dtype == _I64T and slot_mapping.numel() >= T and slot_mapping.is_contiguous()
            and k_cache.is_contiguous() and v_cache.is_contiguous()):
        _cuda(k_cache, v_cache, slot_mapping)
        _refuse("paged_kv_write_fp4",
                (_current(dev, value, k_cache, v_cache, slot_mapping), "tensors must be on the current CUDA device"),
                (H == H2 and value.shape == shape and value.dtype == dtype, "key/value/cache shapes"),
                (dtype in _DTYPES, f"unsupported dtype {dtype}"),
                (False, "slot_mapping: int64 [num_tokens]"))
    ks, kh, k1 = key.stride()
    vs, vh, v1 = value.stride()
    if not (k1 == 1 and v1 == 1 and ((kh == D and vh == D) or H <= 1)):
        _need(False, "key and value: head rows must be dense within a token")
    if T <= 1:   # the stride of a single row says nothing
        ks = vs = H * D
    rc = (_lib or load_library()).pa_paged_kv_write_fp4_strided(
        key.data_ptr(), ks, value.data_ptr(), vs, k_cache.data_ptr(), v_cache.data_ptr(), slot_mapping.data_ptr(), T,
        NB, H, D, PA_BLOCK_SIZE, 0 if dtype == _F16 else 1, float(k_scale), float(v_scale),
        _raw_stream(dev) if stream is None else _stream(stream))
    if rc:
        _check(rc, "pa_paged_kv_write_fp4")


def paged_kv_unpack_fp4(k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: float, v_scale: float,
                        dtype: torch.dtype, stream=None):
    """Both 4-bit pools as 16-bit pools [NB, 16, Hkv, D] of `dtype`."""
    if stream is not None:
        return _given(stream, paged_kv_unpack_fp4, k_cache, v_cache, k_scale, v_scale, dtype)
    NB, H, tile = k_cache.shape
    D = tile // 9
    _fp4_pool(k_cache, v_cache, D)
    dev = k_cache.get_device()
    if not (dev >= 0 and _cuda_device() == dev and v_cache.get_device() == dev and (dtype == _F16 or dtype == _BF16)
            and k_cache.is_contiguous() and v_cache.is_contiguous()):
        _cuda(k_cache, v_cache)
        _refuse("paged_kv_unpack_fp4",
                (_current(dev, v_cache), "tensors must be on the current CUDA device"),
                (False, f"unsupported dtype {dtype}"))
    k_out = torch.empty((NB, PA_BLOCK_SIZE, H, D), dtype=dtype, device=k_cache.device)
    v_out = torch.empty_like(k_out)
    rc = (_lib or load_library()).pa_paged_kv_unpack_fp4(
        k_out.data_ptr(), v_out.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), NB, H, D, PA_BLOCK_SIZE,
        float(k_scale), float(v_scale), 0 if dtype == _F16 else 1, _raw_stream(dev))
    if rc:
        _check(rc, "pa_paged_kv_unpack_fp4")
    return k_out, v_out


def _attn_args(q, k_cache, v_cache, block_tables, seq_lens, cu_q_lens, alibi_slopes, out, workspace, B=None) -> int:
    """What the attention calls below ask of their tensors besides the pools'
    shape (B: the number of sequences, where q does not tell); returns the device."""
    dev = q.get_device()
    if B is None:
        B = q.shape[0] if cu_q_lens is None else seq_lens.shape[0]
    if (dev >= 0 and _cuda_device() == dev and k_cache.get_device() == dev and v_cache.get_device() == dev
            and block_tables.get_device() == dev and seq_lens.get_device() == dev
            and block_tables.dtype == _I32T and seq_lens.dtype == _I32T and seq_lens.numel() == B
            and block_tables.dim() == 2 and block_tables.shape[0] >= B
            and q.is_contiguous() and k_cache.is_contiguous() and v_cache.is_contiguous()
            and block_tables.is_contiguous() and seq_lens.is_contiguous()
            and (q.dtype == _F16 or q.dtype == _BF16)
            and (out is None or (out.get_device() == dev and out.shape == q.shape and out.dtype == q.dtype
                                 and out.is_contiguous()))
            and (cu_q_lens is None or (cu_q_lens.get_device() == dev and cu_q_lens.dtype == _I32T
                                       and cu_q_lens.shape[0] == B + 1 and cu_q_lens.is_contiguous()))
            and (alibi_slopes is None or (alibi_slopes.get_device() == dev and alibi_slopes.dtype == _F32
                                          and alibi_slopes.numel() == q.shape[1] and alibi_slopes.is_contiguous()))
            and (workspace is None or (workspace.get_device() == dev and workspace.is_contiguous()))):
        return dev
    _cuda(q, k_cache, v_cache, block_tables, seq_lens, cu_q_lens, alibi_slopes, out, workspace)
    _refuse("paged attention",
            (_current(dev, k_cache, v_cache, block_tables, seq_lens, cu_q_lens, alibi_slopes, out, workspace),
             "tensors must be on the current CUDA device"),
            (q.dtype in _DTYPES, f"unsupported dtype {q.dtype}"),
            (block_tables.dtype == _I32T and seq_lens.dtype == _I32T, "int32 tables"),
            (seq_lens.numel() == B and block_tables.dim() == 2 and block_tables.shape[0] >= B, "table shapes"),
            (cu_q_lens is None or (cu_q_lens.dtype == _I32T and cu_q_lens.shape[0] == B + 1), "cu_q_lens"),
            (out is None or (out.shape == q.shape and out.dtype == q.dtype), "out shape/dtype"),
            (False, "alibi_slopes: float32 [num_q_heads]"))


def _window(window) -> int:
    """As a C int: past its range, the longest window (no limit) or a negative one (refused)."""
    return max(-2 ** 31, min(int(window), 2 ** 31 - 1))


def _upper(bound) -> int:
    """An upper bound of lengths as a C int: past its range, the largest (no bound) or a negative one (refused)."""
    return max(-2 ** 31, min(int(bound), 2 ** 31 - 1))


def _pool16(q, k_cache, v_cache):
    NB, bs, Hkv, D = k_cache.shape
    if q.shape[2] != D or v_cache.shape != k_cache.shape or k_cache.dtype != q.dtype or v_cache.dtype != q.dtype:
        _need(False, "cache shape/dtype")
    return NB, bs, Hkv


def _ws(nbytes, q, workspace):
    """(address, bytes) of the caller's workspace, or of a new one."""
    if workspace is None or workspace.numel() * workspace.element_size() < nbytes:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    return workspace, workspace.numel() * workspace.element_size()


def paged_attention_decode_fp4(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                               block_tables: torch.Tensor, seq_lens: torch.Tensor, scale: float, k_scale: float,
                               v_scale: float, max_seq_len: int | None = None, out: torch.Tensor | None = None,
                               partition_size: int = 0, workspace: torch.Tensor | None = None,
                               stream=None) -> torch.Tensor:
    """Decode attention over 4-bit pools [NB, Hkv, fp4_tile_bytes(D)]:
    q [B, Hq, D] -> out [B, Hq, D].  partition_size 0 takes the length of
    `decode_partition_for`."""
    if stream is not None:
        return _given(stream, paged_attention_decode_fp4, q, k_cache, v_cache, block_tables, seq_lens, scale,
                      k_scale, v_scale, max_seq_len, out, partition_size, workspace)
    B, Hq, D = q.shape
    NB, Hkv = _fp4_pool(k_cache, v_cache, D)
    dev = _attn_args(q, k_cache, v_cache, block_tables, seq_lens, None, None, out, workspace)
    if max_seq_len is None:
        max_seq_len = int(seq_lens.max().item()) if B else 0
    if out is None:
        out = torch.empty_like(q)
    lib = _lib or load_library()
    if partition_size == 0:
        partition_size = lib.pa_decode_partition_for(B, Hq, Hkv, max_seq_len)
    workspace, ws_bytes = _ws(lib.pa_decode_workspace_bytes(B, Hq, D, max_seq_len, partition_size), q, workspace)
    rc = lib.pa_paged_attention_decode_fp4(
        out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(),
        block_tables.shape[1], seq_lens.data_ptr(), B, max_seq_len, NB, float(scale), float(k_scale),
        float(v_scale), Hq, Hkv, D,
        PA_BLOCK_SIZE, partition_size, workspace.data_ptr(), ws_bytes, 0 if q.dtype == _F16 else 1,
        _raw_stream(dev))
    if rc:
        _check(rc, "pa_paged_attention_decode_fp4")
    return out


def paged_attention_prefill_fp4(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                block_tables: torch.Tensor, seq_lens: torch.Tensor, cu_q_lens: torch.Tensor,
                                scale: float, k_scale: float, v_scale: float, max_q_len: int, max_seq_len: int,
                                out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                                stream=None, chunk_kv_tokens: int | None = None) -> torch.Tensor:
    """Causal varlen attention of new query rows over 4-bit pools (decodes,
    speculative-verify rows and prefill chunks in one call).  `chunk_kv_tokens`
    as in `paged_attention_prefill_fp8`."""
    if stream is not None:
        return _given(stream, paged_attention_prefill_fp4, q, k_cache, v_cache, block_tables, seq_lens, cu_q_lens,
                      scale, k_scale, v_scale, max_q_len, max_seq_len, out, workspace,
                      chunk_kv_tokens=chunk_kv_tokens)
    T, Hq, D = q.shape
    NB, Hkv = _fp4_pool(k_cache, v_cache, D)
    dev = _attn_args(q, k_cache, v_cache, block_tables, seq_lens, cu_q_lens, None, out, workspace)
    B = seq_lens.shape[0]
    if out is None:
        out = torch.empty_like(q)
    lib = _lib or load_library()
    max_blocks = block_tables.shape[1]
    if max_q_len > 8 and B > 0 and T > 0:
        if chunk_kv_tokens is None:
            chunk_kv_tokens = count_chunk_kv_tokens(seq_lens, cu_q_lens)
        nbytes = lib.pa_prefill_fp4_workspace_bytes(B, T, Hq, Hkv, D, max_seq_len, max_blocks, chunk_kv_tokens)
    else:
        nbytes = lib.pa_prefill_mod_workspace_bytes(B, T, Hq, Hkv, D, max_seq_len)
    workspace, ws_bytes = _ws(nbytes, q, workspace)
    rc = lib.pa_paged_attention_prefill_fp4(
        out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(), max_blocks,
        seq_lens.data_ptr(), cu_q_lens.data_ptr(), B, T, max_q_len, max_seq_len, NB, float(scale),
        float(k_scale), float(v_scale), Hq, Hkv, D, PA_BLOCK_SIZE, workspace.data_ptr(), ws_bytes, 0 if q.dtype == _F16 else 1,
        _raw_stream(dev))
    if rc:
        _check(rc, "pa_paged_attention_prefill_fp4")
    return out


# --------------------------------------------------------------------------
# Modified scores (16-bit cache)
# --------------------------------------------------------------------------

def paged_attention_decode_mod(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                               block_tables: torch.Tensor, seq_lens: torch.Tensor, scale: float,
                               max_seq_len: int | None = None, softcap: float = 0.0, window: int = 0,
                               alibi_slopes: torch.Tensor | None = None, out: torch.Tensor | None = None,
                               partition_size: int = 0, workspace: torch.Tensor | None = None,
                               stream=None) -> torch.Tensor:
    """`paged_attention_decode` with modified scores: softcap * tanh(s / softcap)
    when softcap > 0, plus alibi_slopes[h] * (key - query position), over the
    last `window` positions when window > 0.  partition_size 0 takes the length
    of `decode_partition_for`."""
    if stream is not None:
        return _given(stream, paged_attention_decode_mod, q, k_cache, v_cache, block_tables, seq_lens, scale,
                      max_seq_len, softcap, window, alibi_slopes, out, partition_size, workspace)
    B, Hq, D = q.shape
    NB, bs, Hkv = _pool16(q, k_cache, v_cache)
    dev = _attn_args(q, k_cache, v_cache, block_tables, seq_lens, None, alibi_slopes, out, workspace)
    if max_seq_len is None:
        max_seq_len = int(seq_lens.max().item()) if B else 0
    if out is None:
        out = torch.empty_like(q)
    lib = _lib or load_library()
    if partition_size == 0:
        partition_size = lib.pa_decode_partition_for(B, Hq, Hkv, max_seq_len)
    workspace, ws_bytes = _ws(lib.pa_decode_workspace_bytes(B, Hq, D, max_seq_len, partition_size), q, workspace)
    rc = lib.pa_paged_attention_decode_mod(
        out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(),
        block_tables.shape[1], seq_lens.data_ptr(), B, max_seq_len, NB, float(scale), float(softcap), _window(window),
        _ptr(alibi_slopes), Hq, Hkv, D, bs, partition_size, workspace.data_ptr(), ws_bytes, 0 if q.dtype == _F16 else 1,
        _raw_stream(dev))
    if rc:
        _check(rc, "pa_paged_attention_decode_mod")
    return out


def paged_attention_prefill_mod(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                block_tables: torch.Tensor, seq_lens: torch.Tensor, cu_q_lens: torch.Tensor,
                                scale: float, max_q_len: int, max_seq_len: int, softcap: float = 0.0,
                                window: int = 0, alibi_slopes: torch.Tensor | None = None,
                                out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                                stream=None) -> torch.Tensor:
    """`paged_attention_prefill` (decode, verify and chunk rows in one call) with
    modified scores, as `paged_attention_decode_mod`."""
    if stream is not None:
        return _given(stream, paged_attention_prefill_mod, q, k_cache, v_cache, block_tables, seq_lens, cu_q_lens,
                      scale, max_q_len, max_seq_len, softcap, window, alibi_slopes, out, workspace)
    T, Hq, D = q.shape
    NB, bs, Hkv = _pool16(q, k_cache, v_cache)
    dev = _attn_args(q, k_cache, v_cache, block_tables, seq_lens, cu_q_lens, alibi_slopes, out, workspace)
    B = seq_lens.shape[0]
    if out is None:
        out = torch.empty_like(q)
    lib = _lib or load_library()
    workspace, ws_bytes = _ws(lib.pa_prefill_mod_workspace_bytes(B, T, Hq, Hkv, D, max_seq_len), q, workspace)
    rc = lib.pa_paged_attention_prefill_mod(
        out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(),
        block_tables.shape[1], seq_lens.data_ptr(), cu_q_lens.data_ptr(), B, T, max_q_len, max_seq_len, NB, float(scale),
        float(softcap), _window(window), _ptr(alibi_slopes), Hq, Hkv, D, bs, workspace.data_ptr(), ws_bytes, 0 if q.dtype == _F16 else 1,
        _raw_stream(dev))
    if rc:
        _check(rc, "pa_paged_attention_prefill_mod")
    return out


# --------------------------------------------------------------------------
# Cross attention (16-bit cache)
# --------------------------------------------------------------------------

def cross_workspace_bytes(num_seqs: int, num_tokens: int, max_q_len: int) -> int:
    return int(load_library().pa_cross_workspace_bytes(num_seqs, num_tokens, max_q_len))


def paged_cross_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                          block_tables: torch.Tensor, enc_lens: torch.Tensor, scale: float,
                          max_enc_len: int | None = None, cu_q_lens: torch.Tensor | None = None,
                          max_q_len: int | None = None, out: torch.Tensor | None = None,
                          workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Attention of decoder rows q [T, Hq, D] to an encoder's states in a paged
    cache: every row of sequence b sees its enc_lens[b] states (none: a row of
    zeros).  The beams of a request, or a prompt's tokens, are rows of one
    sequence: T / B rows each, or, with cu_q_lens, rows cu_q_lens[b] ..
    cu_q_lens[b + 1] - 1.  max_q_len and max_enc_len are read from the device when
    they are not given; a max_q_len of 8 or less says that there are no longer
    chunks (one that is there all the same is flagged and not written)."""
    if stream is not None:
        return _given(stream, paged_cross_attention, q, k_cache, v_cache, block_tables, enc_lens, scale, max_enc_len,
                      cu_q_lens, max_q_len, out, workspace)
    T, Hq, D = q.shape
    NB, bs, Hkv = _pool16(q, k_cache, v_cache)
    B = enc_lens.shape[0]
    dev = _attn_args(q, k_cache, v_cache, block_tables, enc_lens, cu_q_lens, None, out, workspace, B)
    if cu_q_lens is None:
        if B == 0 or T % B:
            _need(B > 0 and T % B == 0, "without cu_q_lens, q holds the same number of rows for every sequence")
        max_q_len = T // B
    elif max_q_len is None:
        max_q_len = int((cu_q_lens[1:] - cu_q_lens[:-1]).max().item()) if B else 0
    else:
        max_q_len = _upper(max_q_len)
    if max_enc_len is None:
        max_enc_len = int(enc_lens.max().item()) if B else 0
    else:
        max_enc_len = _upper(max_enc_len)
    if out is None:
        out = torch.empty_like(q)
    lib = _lib or load_library()
    ws, ws_bytes = None, 0
    if max_q_len > 8:
        workspace, ws_bytes = _ws(lib.pa_cross_workspace_bytes(B, T, max_q_len), q, workspace)
        ws = workspace.data_ptr()
    rc = lib.pa_paged_cross_attention(
        out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(),
        block_tables.shape[1], enc_lens.data_ptr(), None if cu_q_lens is None else cu_q_lens.data_ptr(), B, T,
        max_q_len, max_enc_len, NB, float(scale), Hq, Hkv, D, bs, ws, ws_bytes, 0 if q.dtype == _F16 else 1,
        _raw_stream(dev))
    if rc:
        _check(rc, "pa_paged_cross_attention")
    return out


# --------------------------------------------------------------------------
# Beam search
# --------------------------------------------------------------------------

_LOGITS = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}
_U8, _BOOL = torch.uint8, torch.bool


def beam_select_workspace_bytes(num_seqs: int, num_beams: int, vocab: int, num_out: int, dtype: torch.dtype) -> int:
    return int(load_library().pa_beam_select_workspace_bytes(num_seqs, num_beams, vocab, num_out, _LOGITS[dtype]))


def beam_select(logits: torch.Tensor, scores: torch.Tensor, num_out: int, finished: torch.Tensor | None = None,
                end_token: int = -1, out=None, workspace: torch.Tensor | None = None, stream=None):
    """The num_out best continuations of every request: candidate (beam w, token
    v) scores scores[s, w] + log_softmax(logits[s * W + w])[v], best first, ties to
    the lowest w * V + v.

    logits [S * W, V] (or [S, W, V]; fp16, bf16 or fp32; rows may be strided),
    scores float32 [S, W] (-inf: a beam without candidates).  `finished` uint8 or
    bool [S, W]: an ended beam's only candidate is end_token, at its own score.
    Returns (scores float32, parents int32, tokens int32), each [S, num_out], and
    with `finished` a fourth like it: the parent had ended, or the token is
    end_token.  `out`: these tensors, to write to (with num_out == W they may be
    scores and finished themselves)."""
    if stream is not None:
        return _given(stream, beam_select, logits, scores, num_out, finished, end_token, out, workspace)
    S, W = scores.shape
    rows, dtype, dev = logits, logits.dtype, logits.get_device()
    if logits.dim() == 3 and logits.shape[:2] == (S, W) and (
            S == 1 or W == 1 or logits.stride(0) == W * logits.stride(1)):
        rows = logits[:, 0] if W == 1 else logits[0] if S == 1 else logits.flatten(0, 1)
    shape = rows.shape
    V = shape[-1]
    num_out, end_token = int(num_out), int(end_token)
    code = _LOGITS.get(dtype)
    ended = _U8 if finished is None else finished.dtype
    if not (dev >= 0 and _cuda_device() == dev and code is not None and len(shape) == 2 and shape[0] == S * W
            and (rows.is_contiguous() or V <= 1 or rows.stride(1) == 1) and 0 < num_out < 2 ** 31
            and scores.get_device() == dev and scores.dtype == _F32 and scores.is_contiguous()
            and (finished is None or (finished.get_device() == dev and finished.shape == scores.shape
                                      and (ended == _U8 or ended == _BOOL) and finished.is_contiguous()
                                      and 0 <= end_token < V))
            and (workspace is None or (workspace.get_device() == dev and workspace.is_contiguous()))):
        _refuse("beam_select",
                (_current(dev, scores, finished, workspace), "tensors must be on the current CUDA device"),
                (code is not None, f"unsupported dtype {dtype}"),
                (len(shape) == 2 and shape[0] == S * W and (V <= 1 or rows.stride(1) == 1),
                 "logits: [S * W, V], or [S, W, V] with evenly spaced rows, dense within a row"),
                (0 < num_out < 2 ** 31, "num_out: at least 1, and an int"),
                (scores.dtype == _F32 and scores.is_contiguous(), "scores: contiguous float32 [S, W]"),
                (finished is None or (finished.shape == scores.shape and (ended == _U8 or ended == _BOOL)
                                      and finished.is_contiguous()), "finished: contiguous uint8 or bool [S, W]"),
                (False, "end_token: a token, with finished"))
    if out is None:
        size, where = (S, num_out), logits.device
        out = (torch.empty(size, dtype=_F32, device=where), torch.empty(size, dtype=_I32T, device=where),
               torch.empty(size, dtype=_I32T, device=where))
        if finished is not None:
            out += (torch.empty(size, dtype=ended, device=where),)
    else:
        out = tuple(out)
        kinds = (_F32, _I32T, _I32T) if finished is None else (_F32, _I32T, _I32T, ended)
        _need(len(out) == len(kinds) and all(t.get_device() == dev and t.shape == (S, num_out) and t.dtype == d
                                             and t.is_contiguous() for t, d in zip(out, kinds)),
              "out: contiguous tensors [S, num_out] of the results' types")
    lib = _lib or load_library()
    nbytes, ws = lib.pa_beam_select_workspace_bytes(S, W, V, num_out, code), None
    if nbytes:
        workspace, nbytes = _ws(nbytes, logits, workspace)
        ws = workspace.data_ptr()
    if finished is None:
        done, over = None, None
    else:
        done, over = finished.data_ptr(), out[3].data_ptr()
    rc = lib.pa_beam_select(
        out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr(), over, rows.data_ptr(),
        rows.stride(0) if S * W > 1 else V, scores.data_ptr(), done, end_token, S, W, V, num_out, code,
        ws, nbytes, _raw_stream(dev))
    if rc:
        _check(rc, "pa_beam_select")
    return out


_PTRS = {}   # number of layers -> type of an array of that many pointers


def _pool_kind(t: torch.Tensor):
    """(kind, num_blocks, num_kv_heads, head_dim) of a pool of any kind."""
    shape, size = t.shape, t.element_size()
    if len(shape) == 4 and size == 2 and shape[1] == PA_BLOCK_SIZE:
        return 0, shape[0], shape[2], shape[3]
    if len(shape) == 4 and size == 1 and shape[2] == PA_BLOCK_SIZE:
        return 1, shape[0], shape[1], shape[3]
    if len(shape) == 3 and size == 1 and shape[2] % 9 == 0:      # 4-bit tiles
        return 2, shape[0], shape[1], shape[2] // 9
    _need(False, "pools: 16-bit [NB, 16, Hkv, D], FP8 [NB, Hkv, 16, D] or 4-bit tiles [NB, Hkv, bytes]")


def beam_reorder(block_tables: torch.Tensor, seq_lens: torch.Tensor, parents: torch.Tensor, k_caches, v_caches,
                 out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Block tables and caches after a selection: row j of request s goes on from
    row parents[s, j] of the same request.

    block_tables int32 [S * W, max_blocks], seq_lens int32 [S * W] (one length for
    all rows of a request), parents int32 [S, W].  Whole blocks are shared; the
    last, partly filled block of every row is its own (also before the call): the
    lowest child of a parent takes over the parent's, the others take those of
    the rows without a child, and the parent's tokens are copied there in every
    pool of k_caches and v_caches (a tensor, or one for each layer; of any kind).
    Entries behind the last token stay with their row.  Returns the new tables,
    in `out`, by default block_tables itself."""
    if stream is not None:
        return _given(stream, beam_reorder, block_tables, seq_lens, parents, k_caches, v_caches, out)
    ks = [k_caches] if isinstance(k_caches, torch.Tensor) else list(k_caches)
    vs = [v_caches] if isinstance(v_caches, torch.Tensor) else list(v_caches)
    pools = ks + vs
    S, W = parents.shape
    dev = block_tables.get_device()
    shape = block_tables.shape
    kind, NB, H, D = _pool_kind(pools[0]) if pools else (0, 2 ** 27 - 1, 1, 64)
    same = len(ks) == len(vs)
    if pools:
        shape0, dtype0 = pools[0].shape, pools[0].dtype
        for t in pools:
            if not (t.shape == shape0 and t.dtype == dtype0 and t.get_device() == dev and t.is_contiguous()):
                same = False
    if out is None:
        out = block_tables
    elif not (out is block_tables or (out.get_device() == dev and out.shape == shape and out.dtype == _I32T
                                      and out.is_contiguous())):
        _need(False, "out: the shape, dtype and device of block_tables")
    if not (same and dev >= 0 and _cuda_device() == dev and len(shape) == 2 and shape[0] == S * W
            and block_tables.dtype == _I32T and block_tables.is_contiguous()
            and seq_lens.get_device() == dev and seq_lens.dtype == _I32T and seq_lens.numel() == S * W
            and seq_lens.is_contiguous()
            and parents.get_device() == dev and parents.dtype == _I32T and parents.is_contiguous()):
        _refuse("beam_reorder",
                (_current(dev, block_tables, seq_lens, parents, *pools), "tensors must be on the current CUDA device"),
                (block_tables.dtype == _I32T and len(shape) == 2 and shape[0] == S * W
                 and block_tables.is_contiguous(), "block_tables: contiguous int32 [S * W, max_blocks]"),
                (seq_lens.dtype == _I32T and seq_lens.numel() == S * W and seq_lens.is_contiguous(),
                 "seq_lens: int32 [S * W]"),
                (parents.dtype == _I32T and parents.is_contiguous(), "parents: contiguous int32 [S, W]"),
                (False, "k_caches and v_caches: as many, contiguous, of one shape and dtype"))
    n = len(ks)
    ptrs = _PTRS.get(n)
    if ptrs is None:
        ptrs = _PTRS[n] = _p * n
    rc = (_lib or load_library()).pa_beam_reorder(
        out.data_ptr(), block_tables.data_ptr(), shape[1], seq_lens.data_ptr(), parents.data_ptr(), S, W,
        ptrs(*[t.data_ptr() for t in ks]), ptrs(*[t.data_ptr() for t in vs]), n, NB, H, D, PA_BLOCK_SIZE, kind,
        _raw_stream(dev))
    if rc:
        _check(rc, "pa_beam_reorder")
    return out
