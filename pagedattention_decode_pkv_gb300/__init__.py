"""Paged-KV hot path for GB300 (sm_103a): thin Python binding of libpkv.so.

Every function here has the name of the C entry point it calls (declared in
include/pkv.h) and only marshals arguments: it checks tensor placement, dtype
and shape, allocates outputs with torch, and passes raw pointers plus the
current CUDA stream.  All computation happens in the library's CUDA kernels;
if libpkv.so has not been built, importing this package fails.

Sources: "Paged KV Cache - AI infra interview lesson" (Walk the Shapes First;
Step 1: slot_mapping and store_kvcache; Step 2: paged_attention_decode) and
"Block-Paged KV Cache" (The three buffers; Element lookup through the block
table; Validating the storage invariants).
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIBRARY_PATH = os.path.join(_HERE, "libpkv.so")

if not os.path.exists(LIBRARY_PATH):
    raise ImportError(
        f"{LIBRARY_PATH} is not built; run `python pagedattention_decode_pkv_gb300/build.py` "
        "(nvcc, sm_103a) first")

_lib = ctypes.CDLL(LIBRARY_PATH)

PKV_OK, PKV_ERR_INVALID_ARG, PKV_ERR_UNSUPPORTED, PKV_ERR_CUDA, PKV_ERR_OUT_OF_RANGE, \
    PKV_ERR_WORKSPACE = range(6)
PKV_F32, PKV_F16, PKV_BF16 = 0, 1, 2
PKV_U32, PKV_U64 = 0, 1
PKV_CACHE_DTYPE, PKV_CACHE_E4M3, PKV_CACHE_INT8 = 0, 1, 2
PKV_ROPE_NONE, PKV_ROPE_LINEAR, PKV_ROPE_NTK, PKV_ROPE_YARN = 0, 1, 2, 3
ERRBIT_SLOT_RANGE, ERRBIT_BLOCK_RANGE, ERRBIT_CONTEXT, ERRBIT_CSR_PAGE, ERRBIT_CSR_PHYS, \
    ERRBIT_SPAN, ERRBIT_TIMEOUT, ERRBIT_NO_BLOCKS, ERRBIT_REF_COUNT = \
    0x01, 0x02, 0x04, 0x08, 0x10, 0x20, 0x40, 0x80, 0x100
_DTYPE = {torch.float32: PKV_F32, torch.float16: PKV_F16, torch.bfloat16: PKV_BF16}

_vp, _i32, _i64, _sz, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
_f64 = ctypes.c_double
_SIGS = {
    "pkv_last_error_string": ([], ctypes.c_char_p),
    "pkv_version": ([], ctypes.c_char_p),
    "pkv_compute_slot_mapping": ([_vp, _i32, _vp, _vp, _vp, _i32, _i32, _i32, _vp, _i64, _vp, _vp], ctypes.c_int),
    "pkv_store_kvcache": ([_vp, _vp, _vp, _vp, _vp, _i64, _i32, _i32, _i64, ctypes.c_int, _vp, _vp], ctypes.c_int),
    "pkv_paged_attention_decode": ([_vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _i32,
                                    _f32, ctypes.c_int, _vp, _sz, _vp, _vp], ctypes.c_int),
    "pkv_paged_attention_decode_append": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32,
                                           _i32, _i32, _i32, _f32, ctypes.c_int, _vp, _sz, _vp, _vp], ctypes.c_int),
    "pkv_paged_attention_decode_static_ws": ([_vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _i32,
                                              _i32, _i32, _f32, ctypes.c_int, _vp, _vp], ctypes.c_int),
    "pkv_paged_attention_decode_workspace_size": ([_i32, _i32, _i32, _i32, _i32, _i32, ctypes.c_int], _sz),
    "pkv_paged_attention_decode_plan": ([_i32, _i32, _i32, _i32, _i32, _i32, ctypes.c_int, _vp, _vp, _vp],
                                        ctypes.c_int),
    "pkv_unpack_block_paged": ([_vp, _vp, _vp, _vp, ctypes.c_int, _vp, _i32, _i64, _i32, _i64, _i32, _i32, _i64,
                                ctypes.c_int, _vp, _vp], ctypes.c_int),
    "pkv_validate_index_buffers": ([_vp, _vp, ctypes.c_int, _i64, _i64, _i64], ctypes.c_int),
    "pkv_validate_quantization_compatibility": ([_i32, _i32, _i32, _i32], ctypes.c_int),
    "pkv_validate_token_ptr": ([_vp, _vp, ctypes.c_int, _i64, _i32, _i64], ctypes.c_int),
    "pkv_validate_block_paged_shape": ([_vp, _i32, _i32, _i32], ctypes.c_int),
    "pkv_block_paged_element_offset": ([_i64, _i64, _i64, _i64, _i32, _i64, _i32, _i32, _vp, _vp, ctypes.c_int,
                                        _i64, _vp], ctypes.c_int),
    "pkv_paged_attention_prefill": ([_vp, _vp, _vp, _vp, _vp, _i32, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32,
                                     _i32, _f32, ctypes.c_int, _vp, _vp], ctypes.c_int),
    "pkv_paged_attention_decode_mod": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_int, _vp, _i32, _vp, _i32,
                                        _i32, _i32, _i32, _i32, _i32, _i32, _f32, _vp, ctypes.c_int, _vp, _sz, _vp,
                                        _vp], ctypes.c_int),
    "pkv_paged_attention_prefill_mod_workspace_size": ([_i32] * 7, _sz),
    "pkv_paged_attention_prefill_mod": ([_vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_int, _vp, _i32, _vp, _vp, _i32, _i32,
                                         _i32, _i32, _i32, _i32, _i32, _f32, _vp, ctypes.c_int, _vp, _sz, _vp, _vp],
                                        ctypes.c_int),
    "pkv_quantize_kvcache_fp8": ([_vp, _vp, _vp, _i32, _i32, _i32, _i32, ctypes.c_int, _vp], ctypes.c_int),
    "pkv_store_kvcache_fp8": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i32, _i32, _i64, _i32, ctypes.c_int, _vp,
                               _vp], ctypes.c_int),
    "pkv_paged_attention_decode_fp8": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _i32,
                                        _i32, _i32, _f32, ctypes.c_int, _vp, _sz, _vp, _vp], ctypes.c_int),
    "pkv_quantize_kvcache_int8": ([_vp, _vp, _vp, _i32, _i32, _i32, _i32, ctypes.c_int, _vp], ctypes.c_int),
    "pkv_store_kvcache_int8": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i32, _i32, _i64, _i32, ctypes.c_int, _vp,
                                _vp], ctypes.c_int),
    "pkv_paged_attention_decode_int8": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _i32,
                                         _i32, _i32, _f32, ctypes.c_int, _vp, _sz, _vp, _vp], ctypes.c_int),
    "pkv_paged_attention_decode_append_fp8": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32,
                                               _i32, _i32, _i32, _i32, _i32, _f32, ctypes.c_int, _vp, _sz, _vp, _vp],
                                              ctypes.c_int),
    "pkv_paged_attention_decode_append_int8": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32,
                                                _i32, _i32, _i32, _i32, _i32, _f32, ctypes.c_int, _vp, _sz, _vp, _vp],
                                               ctypes.c_int),
    "pkv_grow_block_tables_workspace_size": ([_i32, _i32, _i64], _sz),
    "pkv_grow_block_tables": ([_vp, _i32, _vp, _vp, _i32, _i32, _vp, _i32, _vp, _vp, _i64, _vp, _sz, _vp, _vp],
                              ctypes.c_int),
    "pkv_shrink_block_tables": ([_vp, _i32, _vp, _vp, _i32, _i32, _vp, _i32, _vp, _vp], ctypes.c_int),
    "pkv_store_kvcache_int4": ([_vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _i64, _i32, _i32, _i32, _i32, ctypes.c_int,
                                _vp, _vp], ctypes.c_int),
    "pkv_load_kvcache_int4": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i32, _i32, _i32, _i32, ctypes.c_int, _vp, _vp],
                              ctypes.c_int),
    "pkv_rope_frequencies": ([_i32, _f64, ctypes.c_int, _f64, _f64, _f64, _f64, _vp, _vp], ctypes.c_int),
    "pkv_rope_turns": ([_vp, _i32, _vp], ctypes.c_int),
    "pkv_rope_store_kvcache": ([_vp, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _i64, _i32, _i32, _i32, _i64,
                                ctypes.c_int, _vp, _vp], ctypes.c_int),
    "pkv_rope_store_kvcache_int4": ([_vp, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i32,
                                     _i32, _i32, _i32, _i32, ctypes.c_int, _vp, _vp], ctypes.c_int),
    "pkv_paged_attention_decode_int4_workspace_size": ([_i32] * 5, _sz),
    "pkv_paged_attention_decode_int4": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _i32, _i32,
                                         _i32, _f32, _vp, ctypes.c_int, _vp, _sz, _vp, _vp], ctypes.c_int),
    "pkv_paged_attention_prefill_int4_workspace_size": ([_i32] * 8, _sz),
    "pkv_paged_attention_prefill_int4": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _vp, _i32, _i32, _i32, _i32, _i32,
                                          _i32, _i32, _i32, _f32, _vp, ctypes.c_int, _vp, _sz, _vp, _vp], ctypes.c_int),
    "pkv_selftest_wait_timeout": ([_vp, ctypes.c_uint32, _vp], ctypes.c_int),
    "pkv_allocator_create": ([_i32, _i32, _vp], ctypes.c_int),
    "pkv_allocator_destroy": ([_vp], None),
    "pkv_allocator_add_sequence": ([_vp, _i64, _i64, _vp], ctypes.c_int),
    "pkv_allocator_fork": ([_vp, _i64, _i64, _i64], ctypes.c_int),
    "pkv_allocator_append": ([_vp, _i64, _i64, _vp], ctypes.c_int),
    "pkv_allocator_release": ([_vp, _i64], ctypes.c_int),
    "pkv_allocator_block_table": ([_vp, _i64, _vp, _i32, _vp, _vp], ctypes.c_int),
    "pkv_allocator_stats": ([_vp, _vp, _vp, _vp, _vp], ctypes.c_int),
    "pkv_allocator_check": ([_vp], _i32),
}
for _name, (_args, _res) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.argtypes = _args
    _fn.restype = _res


class _ScoreMod(ctypes.Structure):
    """pkv_score_mod"""

    _fields_ = [("softcap", _f32), ("alibi_slopes", _vp), ("key_starts", _vp), ("prefix_lens", _vp)]


class _Rope(ctypes.Structure):
    """pkv_rope"""

    _fields_ = [("turns", _vp), ("amplitude", _f64), ("rotary_dim", _i32), ("interleaved", _i32)]


class PkvError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"pkv status {status}: {message}")
        self.status = status


def _check(status: int):
    if status != PKV_OK:
        raise PkvError(status, _lib.pkv_last_error_string().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dev(*tensors):
    devs = {t.device for t in tensors if t is not None}
    if len(devs) != 1:
        raise ValueError(f"all tensors must be on one CUDA device, got {devs}")
    d = devs.pop()
    if d.type != "cuda":
        raise ValueError("tensors must be CUDA tensors (no CPU path exists)")
    for t in tensors:
        if t is not None and not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
    return d


def _stream(dev, stream):
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    return ctypes.c_void_p(s.cuda_stream)


def _want(t, dtype, name):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


# Leaner marshalling of the calls below that are a few microseconds long on the GPU.
def _device_of(first, *others):
    """The one CUDA device of all tensors given (None: absent), each contiguous."""
    index = first.get_device()
    if index < 0:
        raise ValueError("tensors must be CUDA tensors (no CPU path exists)")
    if not first.is_contiguous():
        raise ValueError("tensors must be contiguous")
    for t in others:
        if t is not None and (t.get_device() != index or not t.is_contiguous()):
            raise ValueError("all tensors must be contiguous and on one CUDA device")
    return first.device


def _addr(t):
    return None if t is None else t.data_ptr()


def _addrs(*tensors):
    return [None if t is None else t.data_ptr() for t in tensors]


# the raw handle alone: a Stream object costs a short call 2 to 4 us
_CURRENT_RAW = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _raw_stream(dev, stream):
    if stream is not None:
        return stream.cuda_stream
    return torch.cuda.current_stream(dev).cuda_stream if _CURRENT_RAW is None else _CURRENT_RAW(dev.index)


def _empty(n, dtype, dev, stream):
    """An uninitialised tensor that belongs to the stream its kernel runs on: what the
    allocator hands out has no pending use there, and a workspace that is freed on return
    is not given to another stream while the kernel still runs."""
    if stream is None:
        return torch.empty(n, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(n, dtype=dtype, device=dev)


def _flag(err_flag):
    if err_flag is not None and err_flag.dtype != torch.int32:
        raise TypeError("err_flag must be int32")
    return _addr(err_flag)


def _call(dev, fn, *args):
    """Calls a library function with `dev` current and raises on its status."""
    if torch.cuda.current_device() == dev.index:
        status = fn(*args)
    else:
        with torch.cuda.device(dev):
            status = fn(*args)
    if status != PKV_OK:
        _check(status)


def pkv_version() -> str:
    return _lib.pkv_version().decode()


def pkv_compute_slot_mapping(block_tables, starts, ends, cu_new, block_size: int, num_blocks: int, *,
                             num_new_tokens: int | None = None, out=None, err_flag=None, stream=None):
    """int32 slot of every position in [starts[b], ends[b]) of every sequence, at cu_new[b]..."""
    dev = _dev(block_tables, starts, ends, cu_new, out, err_flag)
    for t, n in ((block_tables, "block_tables"), (starts, "starts"), (ends, "ends"), (cu_new, "cu_new")):
        _want(t, torch.int32, n)
    if block_tables.dim() != 2:
        raise ValueError("block_tables must be [num_seqs, max_blocks_per_seq]")
    B = block_tables.shape[0]
    if starts.numel() != B or ends.numel() != B or cu_new.numel() != B + 1:
        raise ValueError("starts/ends need num_seqs entries and cu_new num_seqs+1")
    if out is None:
        if num_new_tokens is None:
            num_new_tokens = int(cu_new[-1].item()) if B else 0  # host read: pass num_new_tokens to avoid it
        out = torch.empty(num_new_tokens, dtype=torch.int32, device=dev)
    _want(out, torch.int32, "out")
    with torch.cuda.device(dev):
        _check(_lib.pkv_compute_slot_mapping(_ptr(block_tables), block_tables.shape[1], _ptr(starts), _ptr(ends),
                                             _ptr(cu_new), B, block_size, num_blocks, _ptr(out), out.numel(),
                                             _ptr(err_flag), _stream(dev, stream)))
    return out


def _table_args(block_tables, a, b, ref_counts, names):
    i32 = torch.int32
    if not (block_tables.dtype is i32 and a.dtype is i32 and b.dtype is i32 and ref_counts.dtype is i32):
        for t, n in ((block_tables, "block_tables"), (a, names[0]), (b, names[1]), (ref_counts, "ref_counts")):
            _want(t, i32, n)
    shape = block_tables.shape
    if len(shape) != 2:
        raise ValueError("block_tables must be [num_seqs, max_blocks_per_seq]")
    if a.numel() != shape[0] or b.numel() != shape[0]:
        raise ValueError(f"{names[0]} and {names[1]} need num_seqs entries")
    return shape


def pkv_grow_block_tables(block_tables, starts, ends, ref_counts, block_size: int, *, num_new_tokens: int, cu_new=None,
                          out=None, workspace=None, err_flag=None, stream=None):
    """Sequence b grows from starts[b] to ends[b] positions: its new blocks (the
    lowest free ones, sequences in order) go into block_tables and ref_counts in
    place.  Returns (cu_new [num_seqs + 1], slot_mapping [num_new_tokens]);
    num_new_tokens may be an upper bound (slots past the last position are -1, all
    of them for an empty batch)."""
    dev = _device_of(block_tables, starts, ends, ref_counts, cu_new, out, workspace, err_flag)
    B, max_blocks = _table_args(block_tables, starts, ends, ref_counts, ("starts", "ends"))
    nb = ref_counts.numel()
    if cu_new is None:
        cu_new = _empty(B + 1, torch.int32, dev, stream)
    if out is None:
        out = _empty(num_new_tokens, torch.int32, dev, stream)
    _want_i32(cu_new=cu_new, out=out)
    if cu_new.numel() != B + 1 or out.numel() != num_new_tokens:
        raise ValueError("cu_new needs num_seqs + 1 entries and out num_new_tokens")
    ws = 0 if workspace is not None else _lib.pkv_grow_block_tables_workspace_size(B, nb, num_new_tokens)
    if ws:
        workspace = _empty(ws, torch.uint8, dev, stream)
    _call(dev, _lib.pkv_grow_block_tables, block_tables.data_ptr(), max_blocks, starts.data_ptr(), ends.data_ptr(), B,
          block_size, ref_counts.data_ptr(), nb, cu_new.data_ptr(), out.data_ptr(), num_new_tokens, _addr(workspace),
          0 if workspace is None else workspace.numel() * workspace.element_size(), _flag(err_flag), _raw_stream(dev, stream))
    if not B:  # the library enqueues nothing for an empty batch
        with torch.cuda.stream(stream):  # None: the current one
            cu_new.zero_()
            out.fill_(-1)
    return cu_new, out


def pkv_shrink_block_tables(block_tables, keeps, lens, ref_counts, block_size: int, *, err_flag=None, stream=None):
    """Sequence b goes back from lens[b] to keeps[b] positions: the table entries
    past the kept blocks become -1 and their blocks' counts fall (in place)."""
    dev = _device_of(block_tables, keeps, lens, ref_counts, err_flag)
    B, max_blocks = _table_args(block_tables, keeps, lens, ref_counts, ("keeps", "lens"))
    _call(dev, _lib.pkv_shrink_block_tables, block_tables.data_ptr(), max_blocks, keeps.data_ptr(), lens.data_ptr(), B,
          block_size, ref_counts.data_ptr(), ref_counts.numel(), _flag(err_flag), _raw_stream(dev, stream))


def pkv_store_kvcache(key, value, k_cache, v_cache, slot_mapping, *, err_flag=None, stream=None):
    """In place: k_cache/v_cache rows slot_mapping[i] <- key[i]/value[i]; slot -1 skipped."""
    dev = _dev(key, value, k_cache, v_cache, slot_mapping, err_flag)
    _want(slot_mapping, torch.int32, "slot_mapping")
    if key.dtype not in _DTYPE or not (key.dtype == value.dtype == k_cache.dtype == v_cache.dtype):
        raise TypeError("key, value and caches must share one of float32/float16/bfloat16")
    if k_cache.dim() != 4 or v_cache.shape != k_cache.shape:
        raise ValueError("caches must be [num_blocks, block_size, num_kv_heads, head_dim]")
    nb, bs, H, d = k_cache.shape
    N = slot_mapping.numel()
    if key.shape != (N, H, d) or value.shape != (N, H, d):
        raise ValueError(f"key/value must be [{N}, {H}, {d}]")
    with torch.cuda.device(dev):
        _check(_lib.pkv_store_kvcache(_ptr(key), _ptr(value), _ptr(k_cache), _ptr(v_cache), _ptr(slot_mapping), N,
                                      H, d, nb * bs, _DTYPE[key.dtype], _ptr(err_flag), _stream(dev, stream)))


def pkv_paged_attention_decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                                              max_context_len, dtype) -> int:
    return int(_lib.pkv_paged_attention_decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                                              block_size, max_context_len, _DTYPE[dtype]))


def pkv_paged_attention_decode_plan(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                                    max_context_len, dtype):
    """(tokens per partition, number of partitions, fast path used)."""
    p, n, f = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
    _check(_lib.pkv_paged_attention_decode_plan(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                                                max_context_len, _DTYPE[dtype], ctypes.byref(p), ctypes.byref(n),
                                                ctypes.byref(f)))
    return p.value, n.value, bool(f.value)


def pkv_paged_attention_decode(q, k_cache, v_cache, block_tables, context_lens, scale: float,
                               max_context_len: int, *, out=None, workspace=None, err_flag=None, stream=None):
    """out[b, h] = softmax(scale * q[b, h] . K^T) V over the sequence's paged context."""
    return _decode(q, None, None, k_cache, v_cache, block_tables, context_lens, scale, max_context_len, out,
                   workspace, err_flag, stream)


def pkv_paged_attention_decode_append(q, key, value, k_cache, v_cache, block_tables, context_lens, scale: float,
                                      max_context_len: int, *, out=None, workspace=None, err_flag=None,
                                      stream=None):
    """One decode step: key[b] / value[b] go to the cache row of position
    context_lens[b] - 1, then the attention of pkv_paged_attention_decode runs
    over the whole context (new token included)."""
    return _decode(q, key, value, k_cache, v_cache, block_tables, context_lens, scale, max_context_len, out,
                   workspace, err_flag, stream)


def _decode(q, key, value, k_cache, v_cache, block_tables, context_lens, scale, max_context_len, out, workspace,
            err_flag, stream):
    dev = _dev(q, key, value, k_cache, v_cache, block_tables, context_lens, out, workspace, err_flag)
    if (key is None) != (value is None):
        raise ValueError("key and value go together")
    if key is not None:
        if key.dtype != q.dtype or value.dtype != q.dtype or key.shape != value.shape or \
                key.shape != (q.shape[0], k_cache.shape[2], q.shape[2]) or not key.is_contiguous() or \
                not value.is_contiguous():
            raise ValueError("key, value: contiguous [num_seqs, num_kv_heads, head_dim] of the cache dtype")
    _want(block_tables, torch.int32, "block_tables")
    _want(context_lens, torch.int32, "context_lens")
    if q.dtype not in _DTYPE or not (q.dtype == k_cache.dtype == v_cache.dtype):
        raise TypeError("q and caches must share one of float32/float16/bfloat16")
    if q.dim() != 3 or k_cache.dim() != 4 or v_cache.shape != k_cache.shape or block_tables.dim() != 2:
        raise ValueError("q [B, Hq, d], caches [num_blocks, bs, Hkv, d], block_tables [B, max_blocks]")
    B, Hq, d = q.shape
    nb, bs, Hkv, d2 = k_cache.shape
    if d2 != d or context_lens.numel() != B or block_tables.shape[0] != B:
        raise ValueError("inconsistent shapes")
    if out is None:
        out = torch.empty_like(q)
    ws = pkv_paged_attention_decode_workspace_size(B, Hq, Hkv, d, bs, max_context_len, q.dtype) if B else 0
    if ws and workspace is None:
        workspace = torch.empty(ws, dtype=torch.uint8, device=dev)
    wsp = _ptr(workspace) if ws else None
    wsn = workspace.numel() * workspace.element_size() if ws else 0
    with torch.cuda.device(dev):
        if key is None:
            _check(_lib.pkv_paged_attention_decode(
                _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), block_tables.shape[1],
                _ptr(context_lens), B, Hq, Hkv, d, bs, nb, max_context_len, float(scale), _DTYPE[q.dtype],
                wsp, wsn, _ptr(err_flag), _stream(dev, stream)))
        else:
            _check(_lib.pkv_paged_attention_decode_append(
                _ptr(out), _ptr(q), _ptr(key), _ptr(value), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                block_tables.shape[1], _ptr(context_lens), B, Hq, Hkv, d, bs, nb, max_context_len, float(scale),
                _DTYPE[q.dtype], wsp, wsn, _ptr(err_flag), _stream(dev, stream)))
    return out


_INDEX = {torch.int32: PKV_U32, torch.uint32: PKV_U32, torch.int64: PKV_U64, torch.uint64: PKV_U64}


def pkv_unpack_block_paged(page_pool, block_table, seq_ptr, token_ptr, *, total_tokens: int | None = None,
                           out=None, err_flag=None, stream=None):
    """Contiguous [total_tokens, num_heads, head_dim] of one {kv_role, layer} snapshot."""
    dev = _dev(page_pool, block_table, seq_ptr, token_ptr, out, err_flag)
    if block_table.dtype != seq_ptr.dtype or block_table.dtype not in _INDEX:
        raise TypeError("block_table and seq_ptr must share a 32- or 64-bit integer type")
    _want(token_ptr, torch.int64, "token_ptr")
    if page_pool.dim() != 4 or page_pool.dtype not in _DTYPE:
        raise ValueError("page_pool must be [num_pages, page_size, num_heads, head_dim] float32/16/bf16")
    num_pages, ps, H, d = page_pool.shape
    S = seq_ptr.numel() - 1
    if token_ptr.numel() != S + 1:
        raise ValueError("token_ptr needs num_seqs + 1 entries")
    if out is None:
        if total_tokens is None:
            total_tokens = int(token_ptr[-1].item())  # host read: pass total_tokens to avoid it
        out = torch.empty(total_tokens, H, d, dtype=page_pool.dtype, device=dev)
    shape = (ctypes.c_int64 * out.dim())(*out.shape)
    _check(_lib.pkv_validate_block_paged_shape(shape, out.dim(), H, d))
    with torch.cuda.device(dev):
        _check(_lib.pkv_unpack_block_paged(_ptr(out), _ptr(page_pool), _ptr(block_table), _ptr(seq_ptr),
                                           _INDEX[block_table.dtype], _ptr(token_ptr), S, block_table.numel(), ps,
                                           num_pages, H, d, out.shape[0], _DTYPE[page_pool.dtype], _ptr(err_flag),
                                           _stream(dev, stream)))
    return out


def _host_index(x, dtype=None):
    t = torch.as_tensor(x)
    if dtype is not None:
        t = t.to(dtype)
    elif t.dtype not in _INDEX:
        t = t.to(torch.int64)
    return t.cpu().contiguous()


def pkv_validate_index_buffers(seq_ptr, block_table, num_pages: int, index_dtype=None):
    """Raises PkvError unless the page's four storage invariants hold (host data)."""
    sp = _host_index(seq_ptr, index_dtype)
    bt = _host_index(block_table, sp.dtype)
    _check(_lib.pkv_validate_index_buffers(_ptr(sp), _ptr(bt) if bt.numel() else None, _INDEX[sp.dtype],
                                           sp.numel() - 1, bt.numel(), num_pages))


QUANT_NONE, QUANT_PER_TENSOR, QUANT_PER_CHANNEL, QUANT_PER_BLOCK = 0x00, 0x01, 0x02, 0x03


def pkv_validate_quantization_compatibility(scheme_tag: int, axis: int, block_size: int, page_size: int):
    """Raises PkvError unless the scheme's scales fit the block-paged layout:
    per-block-affine along the paged axis (0) with block_size == page_size;
    per-channel not along the paged axis."""
    _check(_lib.pkv_validate_quantization_compatibility(scheme_tag, axis, block_size, page_size))


def pkv_validate_token_ptr(token_ptr, seq_ptr, page_size: int, total_tokens: int, index_dtype=None):
    tp = _host_index(token_ptr, torch.int64)
    sp = _host_index(seq_ptr, index_dtype)
    _check(_lib.pkv_validate_token_ptr(_ptr(tp), _ptr(sp), _INDEX[sp.dtype], sp.numel() - 1, page_size,
                                       total_tokens))


def pkv_validate_block_paged_shape(shape, num_heads: int, head_dim: int):
    arr = (ctypes.c_int64 * max(1, len(shape)))(*shape)
    _check(_lib.pkv_validate_block_paged_shape(arr, len(shape), num_heads, head_dim))


def pkv_block_paged_element_offset(seq, token, head, dim, page_size, num_pages, num_heads, head_dim,
                                   block_table, seq_ptr, index_dtype=None) -> int:
    sp = _host_index(seq_ptr, index_dtype)
    bt = _host_index(block_table, sp.dtype)
    flat = ctypes.c_int64()
    _check(_lib.pkv_block_paged_element_offset(seq, token, head, dim, page_size, num_pages, num_heads, head_dim,
                                               _ptr(bt), _ptr(sp), _INDEX[sp.dtype], sp.numel() - 1,
                                               ctypes.byref(flat)))
    return flat.value


def pkv_paged_attention_prefill(q, k_cache, v_cache, block_tables, starts, cu_q, scale: float, max_q_len: int, *,
                                out=None, err_flag=None, stream=None):
    """Causal prefill: query i of sequence b (row cu_q[b] + i of q, position
    starts[b] + i) attends over positions 0 .. starts[b] + i of its paged context."""
    dev = _dev(q, k_cache, v_cache, block_tables, starts, cu_q, out, err_flag)
    _want(block_tables, torch.int32, "block_tables")
    _want(starts, torch.int32, "starts")
    _want(cu_q, torch.int32, "cu_q")
    if q.dtype not in _DTYPE or not (q.dtype == k_cache.dtype == v_cache.dtype):
        raise TypeError("q and caches must share one of float32/float16/bfloat16")
    Tq, Hq, d = q.shape
    nb, bs, Hkv, _ = k_cache.shape
    B = starts.numel()
    if cu_q.numel() != B + 1 or block_tables.shape[0] != B:
        raise ValueError("inconsistent shapes")
    if out is None:
        out = torch.empty_like(q)
    with torch.cuda.device(dev):
        _check(_lib.pkv_paged_attention_prefill(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                                block_tables.shape[1], _ptr(starts), _ptr(cu_q), B, max_q_len, Hq,
                                                Hkv, d, bs, nb, float(scale), _DTYPE[q.dtype], _ptr(err_flag),
                                                _stream(dev, stream)))
    return out


# ----------------------------------------------------------------------------- score rules, any cache format
_FORMAT = {torch.uint8: PKV_CACHE_E4M3, torch.int8: PKV_CACHE_INT8}


def _cache_format(q, k_cache, v_cache, k_scale, v_scale):
    """(pkv_cache_format, q's shape, the caches' shape), with types, shapes and scales checked."""
    dtype, code, q_shape, shape = q.dtype, k_cache.dtype, q.shape, k_cache.shape
    if dtype not in _DTYPE or v_cache.dtype is not code:
        raise TypeError("q must be float32/float16/bfloat16 and both caches of one type")
    if len(q_shape) != 3 or len(shape) != 4 or v_cache.shape != shape or shape[3] != q_shape[2]:
        raise ValueError("q [rows, Hq, d], caches [num_blocks, bs, Hkv, d]")
    fmt = _FORMAT.get(code, PKV_CACHE_DTYPE)
    if fmt == PKV_CACHE_DTYPE:
        if code is not dtype:
            raise TypeError("caches must have the type of q, uint8 (E4M3 codes) or int8")
        if k_scale is not None or v_scale is not None:
            raise ValueError("scales belong to 8-bit caches")
    else:
        for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if t is None:
                raise ValueError(f"{name} is required for an 8-bit cache")
            _want(t, torch.float32, name)
            if t.shape != (shape[0], shape[2]):
                raise ValueError(f"{name} must be [num_blocks, num_kv_heads]")
    return fmt, q_shape, shape


def _want_i32(**tensors):
    for name, t in tensors.items():
        if t.dtype is not torch.int32:
            raise TypeError(f"{name} must be torch.int32")


def _score_mod(softcap, alibi_slopes, key_starts, prefix_lens, Hq, rows, B):
    """A pkv_score_mod by reference, None for plain causal attention."""
    if alibi_slopes is not None and (alibi_slopes.dtype is not torch.float32 or alibi_slopes.numel() != Hq):
        raise ValueError(f"alibi_slopes: {Hq} entries of torch.float32")
    if key_starts is not None and (key_starts.dtype is not torch.int32 or key_starts.numel() != rows):
        raise ValueError(f"key_starts: {rows} entries of torch.int32")
    if prefix_lens is not None and (prefix_lens.dtype is not torch.int32 or prefix_lens.numel() != B):
        raise ValueError(f"prefix_lens: {B} entries of torch.int32")
    if softcap == 0 and alibi_slopes is None and key_starts is None and prefix_lens is None:
        return None
    return ctypes.byref(_ScoreMod(softcap, *_addrs(alibi_slopes, key_starts, prefix_lens)))


def pkv_paged_attention_decode_mod(q, k_cache, v_cache, block_tables, context_lens, scale: float,
                                   max_context_len: int, *, key=None, value=None, softcap: float = 0.0,
                                   alibi_slopes=None, key_starts=None, k_scale=None, v_scale=None, out=None,
                                   workspace=None, err_flag=None, stream=None):
    """Decode attention with score rules, over caches of q's type or of 8-bit codes
    (uint8 E4M3 or int8, with k_scale / v_scale): softcap * tanh(s / softcap), minus
    alibi_slopes[h] * (query - key position); sequence b sees keys from
    key_starts[b] on.  With key / value the step's new row is appended first."""
    dev = _device_of(q, key, value, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, alibi_slopes, key_starts,
               out, workspace, err_flag)
    fmt, (B, Hq, d), (nb, bs, Hkv, _) = _cache_format(q, k_cache, v_cache, k_scale, v_scale)
    _want_i32(block_tables=block_tables, context_lens=context_lens)
    tables = block_tables.shape
    if context_lens.numel() != B or len(tables) != 2 or tables[0] != B:
        raise ValueError("inconsistent shapes")
    if (key is None) != (value is None):
        raise ValueError("key and value go together")
    if key is not None and not (key.dtype == value.dtype == q.dtype and key.shape == value.shape == (B, Hkv, d)):
        raise ValueError("key, value: [num_seqs, num_kv_heads, head_dim] of the q dtype")
    mod = _score_mod(softcap, alibi_slopes, key_starts, None, Hq, B, B)
    if out is None:
        out = _empty((B, Hq, d), q.dtype, dev, stream)
    elif out.shape != q.shape or out.dtype != q.dtype:
        raise ValueError("out must have the shape and type of q")
    dtype = _DTYPE[q.dtype]
    ws = _lib.pkv_paged_attention_decode_workspace_size(B, Hq, Hkv, d, bs, max_context_len, dtype) if B else 0
    if ws and workspace is None:
        workspace = _empty(ws, torch.uint8, dev, stream)
    _call(dev, _lib.pkv_paged_attention_decode_mod,
          *_addrs(out, q, key, value, k_cache, v_cache, k_scale, v_scale), fmt, block_tables.data_ptr(), tables[1],
          context_lens.data_ptr(), B, Hq, Hkv, d, bs, nb, max_context_len, scale, mod, dtype,
          workspace.data_ptr() if ws else None, workspace.numel() * workspace.element_size() if ws else 0,
          _flag(err_flag), _raw_stream(dev, stream))
    return out


def pkv_paged_attention_prefill_mod_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                                                   max_q_len, max_blocks_per_seq) -> int:
    return int(_lib.pkv_paged_attention_prefill_mod_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                                                   block_size, max_q_len, max_blocks_per_seq))


def pkv_paged_attention_prefill_mod(q, k_cache, v_cache, block_tables, starts, cu_q, scale: float, max_q_len: int, *,
                                    softcap: float = 0.0, alibi_slopes=None, key_starts=None, prefix_lens=None,
                                    k_scale=None, v_scale=None, out=None, workspace=None, err_flag=None, stream=None):
    """Prefill attention with score rules, over caches of q's type or of 8-bit codes
    (uint8 E4M3 or int8, with k_scale / v_scale): softcap * tanh(s / softcap), minus
    alibi_slopes[h] * |p - t|; query row i sees keys key_starts[i] <= t <= p, and
    those below prefix_lens[b]."""
    dev = _device_of(q, k_cache, v_cache, k_scale, v_scale, block_tables, starts, cu_q, alibi_slopes, key_starts,
               prefix_lens, out, workspace, err_flag)
    fmt, (rows, Hq, d), (nb, bs, Hkv, _) = _cache_format(q, k_cache, v_cache, k_scale, v_scale)
    _want_i32(block_tables=block_tables, starts=starts, cu_q=cu_q)
    B, tables = starts.numel(), block_tables.shape
    if cu_q.numel() != B + 1 or len(tables) != 2 or tables[0] != B:
        raise ValueError("inconsistent shapes")
    mod = _score_mod(softcap, alibi_slopes, key_starts, prefix_lens, Hq, rows, B)
    if out is None:
        out = _empty((rows, Hq, d), q.dtype, dev, stream)
    elif out.shape != q.shape or out.dtype != q.dtype:
        raise ValueError("out must have the shape and type of q")
    ws = _lib.pkv_paged_attention_prefill_mod_workspace_size(B, Hq, Hkv, d, bs, max_q_len, tables[1])
    if ws and workspace is None:
        workspace = _empty(ws, torch.uint8, dev, stream)
    _call(dev, _lib.pkv_paged_attention_prefill_mod, *_addrs(out, q, k_cache, v_cache, k_scale, v_scale), fmt,
          block_tables.data_ptr(), tables[1], starts.data_ptr(), cu_q.data_ptr(), B, max_q_len, Hq, Hkv, d, bs, nb, scale,
          mod, _DTYPE[q.dtype], workspace.data_ptr() if ws else None,
          workspace.numel() * workspace.element_size() if ws else 0, _flag(err_flag), _raw_stream(dev, stream))
    return out


# ----------------------------------------------------------------------------- 8-bit (E4M3 / int8) caches
# Code caches: E4M3 as torch.uint8 bytes, int8 as torch.int8.
_CODES = {"fp8": torch.uint8, "int8": torch.int8}


def _quantize_codes(fmt, cache, codes, scales, stream):
    dev = _dev(cache, codes, scales)
    if cache.dtype not in _DTYPE or cache.dim() != 4:
        raise ValueError("cache: [num_blocks, bs, Hkv, d] of float32/float16/bfloat16")
    nb, bs, H, d = cache.shape
    if codes is None:
        codes = torch.empty(cache.shape, dtype=_CODES[fmt], device=dev)
    if scales is None:
        scales = torch.empty(nb, H, dtype=torch.float32, device=dev)
    _want(codes, _CODES[fmt], "codes")
    _want(scales, torch.float32, "scales")
    fn = getattr(_lib, "pkv_quantize_kvcache_" + fmt)
    with torch.cuda.device(dev):
        _check(fn(_ptr(cache), _ptr(codes), _ptr(scales), nb, bs, H, d, _DTYPE[cache.dtype], _stream(dev, stream)))
    return codes, scales


def _store_codes(fmt, key, value, k_cache, v_cache, k_scale, v_scale, slot_mapping, err_flag, stream):
    dev = _dev(key, value, k_cache, v_cache, k_scale, v_scale, slot_mapping, err_flag)
    _want(slot_mapping, torch.int32, "slot_mapping")
    _want(k_cache, _CODES[fmt], "k_cache")
    _want(v_cache, _CODES[fmt], "v_cache")
    nb, bs, H, d = k_cache.shape
    fn = getattr(_lib, "pkv_store_kvcache_" + fmt)
    with torch.cuda.device(dev):
        _check(fn(_ptr(key), _ptr(value), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale),
                  _ptr(slot_mapping), slot_mapping.numel(), H, d, nb * bs, bs, _DTYPE[key.dtype], _ptr(err_flag),
                  _stream(dev, stream)))


def _attention_codes(fmt, q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, scale,
                     max_context_len, out, workspace, err_flag, stream, key=None, value=None):
    dev = _dev(q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, out, workspace, err_flag, key,
               value)
    _want(k_cache, _CODES[fmt], "k_cache")
    _want(v_cache, _CODES[fmt], "v_cache")
    _want(k_scale, torch.float32, "k_scale")
    _want(v_scale, torch.float32, "v_scale")
    _want(block_tables, torch.int32, "block_tables")
    _want(context_lens, torch.int32, "context_lens")
    B, Hq, d = q.shape
    nb, bs, Hkv, _ = k_cache.shape
    if out is None:
        out = torch.empty_like(q)
    ws = pkv_paged_attention_decode_workspace_size(B, Hq, Hkv, d, bs, max_context_len, q.dtype) if B else 0
    if ws and workspace is None:
        workspace = torch.empty(ws, dtype=torch.uint8, device=dev)
    tail = (block_tables.shape[1], _ptr(context_lens), B, Hq, Hkv, d, bs, nb, max_context_len, float(scale),
            _DTYPE[q.dtype], _ptr(workspace) if ws else None,
            workspace.numel() * workspace.element_size() if ws else 0, _ptr(err_flag), _stream(dev, stream))
    with torch.cuda.device(dev):
        if key is None:
            fn = getattr(_lib, "pkv_paged_attention_decode_" + fmt)
            _check(fn(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale),
                      _ptr(block_tables), *tail))
        else:
            if key.dtype != q.dtype or value.dtype != q.dtype or key.shape != (B, Hkv, d) or value.shape != key.shape:
                raise ValueError("key/value must be [num_seqs, num_kv_heads, head_dim] of the q dtype")
            fn = getattr(_lib, "pkv_paged_attention_decode_append_" + fmt)
            _check(fn(_ptr(out), _ptr(q), _ptr(key), _ptr(value), _ptr(k_cache),
                      _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), _ptr(block_tables), *tail))
    return out


def pkv_quantize_kvcache_fp8(cache, *, codes=None, scales=None, stream=None):
    """[num_blocks, bs, Hkv, d] cache -> (uint8 E4M3 codes of the same shape,
    float32 scales [num_blocks, Hkv]); per (block, head) s = max|x| / 448."""
    return _quantize_codes("fp8", cache, codes, scales, stream)


def pkv_store_kvcache_fp8(key, value, k_cache, v_cache, k_scale, v_scale, slot_mapping, *, err_flag=None,
                          stream=None):
    """Writes encode(key[i] / s) into row slot_mapping[i] of the E4M3 code caches (in place)."""
    _store_codes("fp8", key, value, k_cache, v_cache, k_scale, v_scale, slot_mapping, err_flag, stream)


def pkv_paged_attention_decode_fp8(q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens,
                                   scale: float, max_context_len: int, *, out=None, workspace=None, err_flag=None,
                                   stream=None):
    """Decode attention over E4M3 code caches with per-(block, head) scales."""
    return _attention_codes("fp8", q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, scale,
                            max_context_len, out, workspace, err_flag, stream)


def pkv_paged_attention_decode_append_fp8(q, key, value, k_cache, v_cache, k_scale, v_scale, block_tables,
                                          context_lens, scale: float, max_context_len: int, *, out=None,
                                          workspace=None, err_flag=None, stream=None):
    """One decode step over E4M3 code caches: key[b] / value[b] are encoded
    under the existing (block, head) scales into the row of position
    context_lens[b] - 1 (in place), then the attention of
    pkv_paged_attention_decode_fp8 runs over the whole context."""
    return _attention_codes("fp8", q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, scale,
                            max_context_len, out, workspace, err_flag, stream, key, value)


def pkv_quantize_kvcache_int8(cache, *, codes=None, scales=None, stream=None):
    """[num_blocks, bs, Hkv, d] cache -> (int8 codes of the same shape, float32
    scales [num_blocks, Hkv]); per (block, head) s = max|x| / 127."""
    return _quantize_codes("int8", cache, codes, scales, stream)


def pkv_store_kvcache_int8(key, value, k_cache, v_cache, k_scale, v_scale, slot_mapping, *, err_flag=None,
                           stream=None):
    """Writes encode(key[i] / s) into row slot_mapping[i] of the int8 code caches (in place)."""
    _store_codes("int8", key, value, k_cache, v_cache, k_scale, v_scale, slot_mapping, err_flag, stream)


def pkv_paged_attention_decode_int8(q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens,
                                    scale: float, max_context_len: int, *, out=None, workspace=None, err_flag=None,
                                    stream=None):
    """Decode attention over int8 code caches with per-(block, head) scales."""
    return _attention_codes("int8", q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, scale,
                            max_context_len, out, workspace, err_flag, stream)


def pkv_paged_attention_decode_append_int8(q, key, value, k_cache, v_cache, k_scale, v_scale, block_tables,
                                           context_lens, scale: float, max_context_len: int, *, out=None,
                                           workspace=None, err_flag=None, stream=None):
    """One decode step over int8 code caches (see pkv_paged_attention_decode_append_fp8)."""
    return _attention_codes("int8", q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, scale,
                            max_context_len, out, workspace, err_flag, stream, key, value)


# ----------------------------------------------------------------------------- rotary positions, 4-bit caches
class RopeFrequencies:
    """What a model's rotary positions are computed from: `turns`, int64 [rotary_dim / 2] on
    the device (turns per position, 64-bit fixed point), and `amplitude`."""

    def __init__(self, turns, amplitude: float = 1.0):
        _want(turns, torch.int64, "turns")
        if turns.dim() != 1:
            raise ValueError("turns must be [rotary_dim / 2]")
        self.turns, self.amplitude, self.rotary_dim = turns, float(amplitude), 2 * turns.numel()

    def inverse(self):
        """Frequencies that turn back."""
        return RopeFrequencies(-self.turns, 1 / self.amplitude)


_ROPE_SCALING = {None: PKV_ROPE_NONE, "linear": PKV_ROPE_LINEAR, "ntk": PKV_ROPE_NTK, "yarn": PKV_ROPE_YARN}


def pkv_rope_frequencies(rotary_dim: int, base: float = 10000.0, *, scaling=None, factor: float = 1.0, original_len=0,
                         beta_fast: float = 32.0, beta_slow: float = 1.0, device="cuda") -> RopeFrequencies:
    """Frequencies base^(-2 i / rotary_dim); `scaling` "linear", "ntk" or "yarn" stretches them
    for contexts `factor` times as long (yarn: as `original_len`)."""
    if scaling not in _ROPE_SCALING:
        raise ValueError(f"scaling must be one of {list(_ROPE_SCALING)}")
    turns, amplitude = torch.empty(max(rotary_dim, 0) // 2, dtype=torch.int64), ctypes.c_double()
    _check(_lib.pkv_rope_frequencies(rotary_dim, base, _ROPE_SCALING[scaling], factor, original_len, beta_fast, beta_slow,
                                     _ptr(turns), ctypes.byref(amplitude)))
    return RopeFrequencies(turns.to(device), amplitude.value)


def pkv_rope_turns(inv_freq, *, amplitude: float = 1.0, device="cuda") -> RopeFrequencies:
    """Frequencies given as radians per position (a sequence or a tensor, [rotary_dim / 2])."""
    f = torch.as_tensor(inv_freq, dtype=torch.float64).detach().cpu().contiguous()
    turns = torch.empty(f.shape, dtype=torch.int64)
    _check(_lib.pkv_rope_turns(_ptr(f), f.numel(), _ptr(turns)))
    return RopeFrequencies(turns.to(device), amplitude)


def _heads(x, h, d, index, name):
    """Elements between the tokens of x [tokens, h, d], whose heads and dims are contiguous."""
    if x.get_device() != index:
        raise ValueError("all tensors must be on one CUDA device")
    n, a, b = x.stride()
    if (b != 1 and d > 1) or (a != d and h > 1):
        if x.numel():
            raise ValueError(f"{name}: the heads of a token must be contiguous")
    return n if x.shape[0] > 1 else h * d


def _int4_cache(k_cache, v_cache, k_scale, v_scale):
    """(num_blocks, Hkv, block_size, d) of 4-bit caches, checked."""
    shape, scales = k_cache.shape, k_scale.shape
    if k_cache.dtype is not torch.uint8 or v_cache.dtype is not torch.uint8:
        raise TypeError("k_cache and v_cache must be torch.uint8 (two codes a byte)")
    if k_scale.dtype is not torch.float16 or v_scale.dtype is not torch.float16:
        raise TypeError("k_scale and v_scale must be torch.float16")
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError("k_cache, v_cache: [num_blocks, Hkv, bs, head_dim / 2]")
    nb, H, bs, half = shape
    if scales != (nb, H, bs, half // 16) or v_scale.shape != scales:
        raise ValueError("k_scale, v_scale: [num_blocks, Hkv, bs, head_dim / 32]")
    return nb, H, bs, 2 * half


def _rope_store(fn, H, d, tail, q, key, value, positions, rope, caches, slot_mapping, interleaved, out, err_flag, stream):
    """The marshalling of the store calls; q, and with it positions and rope, may be absent."""
    dtype, n = key.dtype, slot_mapping.numel()
    if dtype not in _DTYPE or value.dtype is not dtype:
        raise TypeError("key and value must share one of float32/float16/bfloat16")
    if slot_mapping.dtype is not torch.int32:
        raise TypeError("slot_mapping must be torch.int32")
    rows = (n, H, d)
    if key.shape != rows or value.shape != rows:
        raise ValueError(f"key/value must be [{n}, {H}, {d}]")
    if q is None:
        dev = _device_of(slot_mapping, *caches, err_flag)
        index = dev.index
        front = (key.data_ptr(), _heads(key, H, d, index, "key"), value.data_ptr(), _heads(value, H, d, index, "value"))
    else:
        turns, shape = rope.turns, q.shape
        dev = _device_of(slot_mapping, *caches, positions, turns, out, err_flag)
        index = dev.index
        if q.dtype is not dtype:
            raise TypeError("q must have the type of key and value")
        if len(shape) != 3 or shape[0] != n or shape[2] != d:
            raise ValueError(f"q must be [{n}, Hq, {d}]")
        if positions.dtype is not torch.int32 or positions.numel() != n:
            raise ValueError(f"positions: {n} entries of torch.int32")
        if out is None:
            out = _empty(shape, dtype, dev, stream)
        elif out.shape != shape or out.dtype is not dtype:
            raise ValueError("out must have the shape and type of q")
        Hq = shape[1]
        front = (out.data_ptr(), q.data_ptr(), _heads(q, Hq, d, index, "q"), key.data_ptr(), _heads(key, H, d, index, "key"),
                 value.data_ptr(), _heads(value, H, d, index, "value"), positions.data_ptr(),
                 ctypes.byref(_Rope(turns.data_ptr(), rope.amplitude, rope.rotary_dim, 1 if interleaved else 0)))
        tail = (Hq, *tail)
    _call(dev, fn, *front, *[t.data_ptr() for t in caches], slot_mapping.data_ptr(), n, *tail, _DTYPE[dtype], _flag(err_flag),
          _raw_stream(dev, stream))
    return out


def pkv_rope_store_kvcache(q, key, value, positions, rope: RopeFrequencies, k_cache, v_cache, slot_mapping, *,
                           interleaved: bool = False, out=None, err_flag=None, stream=None):
    """Rotates q and key by their positions: the queries are returned (into `out`, which may be
    q itself), row slot_mapping[i] of the caches receives the rotated key[i] and value[i] (slot
    -1 skipped).  q, key and value may be parts of one projection's output."""
    shape = k_cache.shape
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError("caches must be [num_blocks, block_size, num_kv_heads, head_dim]")
    if k_cache.dtype is not key.dtype or v_cache.dtype is not key.dtype:
        raise TypeError("key, value and caches must share one type")
    nb, bs, H, d = shape
    return _rope_store(_lib.pkv_rope_store_kvcache, H, d, (H, d, nb * bs), q, key, value, positions, rope,
                       (k_cache, v_cache), slot_mapping, interleaved, out, err_flag, stream)


def pkv_rope_store_kvcache_int4(q, key, value, positions, rope: RopeFrequencies, k_cache, v_cache, k_scale, v_scale,
                                slot_mapping, *, interleaved: bool = False, out=None, err_flag=None, stream=None):
    """pkv_rope_store_kvcache into 4-bit caches (uint8 [num_blocks, Hkv, bs, head_dim / 2] with
    float16 scales [num_blocks, Hkv, bs, head_dim / 32])."""
    nb, H, bs, d = _int4_cache(k_cache, v_cache, k_scale, v_scale)
    return _rope_store(_lib.pkv_rope_store_kvcache_int4, H, d, (H, d, bs, nb), q, key, value, positions, rope,
                       (k_cache, v_cache, k_scale, v_scale), slot_mapping, interleaved, out, err_flag, stream)


def pkv_store_kvcache_int4(key, value, k_cache, v_cache, k_scale, v_scale, slot_mapping, *, err_flag=None, stream=None):
    """Row slot_mapping[i] of the 4-bit caches <- key[i] / value[i], each 32 dims under their own
    scale (in place; slot -1 skipped)."""
    nb, H, bs, d = _int4_cache(k_cache, v_cache, k_scale, v_scale)
    _rope_store(_lib.pkv_store_kvcache_int4, H, d, (H, d, bs, nb), None, key, value, None, None,
                (k_cache, v_cache, k_scale, v_scale), slot_mapping, False, None, err_flag, stream)


def pkv_load_kvcache_int4(k_cache, v_cache, k_scale, v_scale, slot_mapping, dtype=torch.float16, *, out=None, err_flag=None,
                          stream=None):
    """(key, value) [num_tokens, Hkv, head_dim] of `dtype`: the rows slot_mapping of the 4-bit
    caches read back (slot -1: zeros)."""
    nb, H, bs, d = _int4_cache(k_cache, v_cache, k_scale, v_scale)
    if dtype not in _DTYPE:
        raise TypeError("dtype must be float32/float16/bfloat16")
    if slot_mapping.dtype is not torch.int32:
        raise TypeError("slot_mapping must be torch.int32")
    n = slot_mapping.numel()
    key, value = out if out is not None else (None, None)
    dev = _device_of(k_cache, v_cache, k_scale, v_scale, slot_mapping, key, value, err_flag)
    if out is None:
        key, value = _empty((n, H, d), dtype, dev, stream), _empty((n, H, d), dtype, dev, stream)
    elif not (key.shape == value.shape == (n, H, d) and key.dtype == value.dtype == dtype):
        raise ValueError(f"out must be two tensors [{n}, {H}, {d}] of dtype")
    _call(dev, _lib.pkv_load_kvcache_int4, key.data_ptr(), value.data_ptr(), *_addrs(k_cache, v_cache, k_scale, v_scale),
          slot_mapping.data_ptr(), n, H, d, bs, nb, _DTYPE[dtype], _flag(err_flag), _raw_stream(dev, stream))
    return key, value


def pkv_paged_attention_decode_int4_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, max_context_len) -> int:
    return int(_lib.pkv_paged_attention_decode_int4_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                                                   max_context_len))


def pkv_paged_attention_decode_int4(q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, scale: float,
                                    max_context_len: int, *, softcap: float = 0.0, alibi_slopes=None, key_starts=None,
                                    out=None, workspace=None, err_flag=None, stream=None):
    """Decode attention over 4-bit caches (as pkv_store_kvcache_int4 writes them), with the score
    rules of pkv_paged_attention_decode_mod."""
    nb, Hkv, bs, d = _int4_cache(k_cache, v_cache, k_scale, v_scale)
    dev = _device_of(q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, alibi_slopes, key_starts, out,
                     workspace, err_flag)
    dtype, shape, tables = q.dtype, q.shape, block_tables.shape
    if dtype not in _DTYPE:
        raise TypeError("q must be float16/bfloat16")
    if len(shape) != 3 or shape[2] != d:
        raise ValueError(f"q must be [num_seqs, Hq, {d}]")
    B, Hq = shape[0], shape[1]
    _want_i32(block_tables=block_tables, context_lens=context_lens)
    if context_lens.numel() != B or len(tables) != 2 or tables[0] != B:
        raise ValueError("inconsistent shapes")
    mod = _score_mod(softcap, alibi_slopes, key_starts, None, Hq, B, B)
    if out is None:
        out = _empty(shape, dtype, dev, stream)
    elif out.shape != shape or out.dtype is not dtype:
        raise ValueError("out must have the shape and type of q")
    ws = _lib.pkv_paged_attention_decode_int4_workspace_size(B, Hq, Hkv, d, max_context_len)
    if ws and workspace is None:
        workspace = _empty(ws, torch.uint8, dev, stream)
    _call(dev, _lib.pkv_paged_attention_decode_int4, *_addrs(out, q, k_cache, v_cache, k_scale, v_scale),
          block_tables.data_ptr(), tables[1], context_lens.data_ptr(), B, Hq, Hkv, d, bs, nb, max_context_len, scale, mod,
          _DTYPE[dtype], workspace.data_ptr() if ws else None, workspace.numel() * workspace.element_size() if ws else 0,
          _flag(err_flag), _raw_stream(dev, stream))
    return out


def pkv_paged_attention_prefill_int4_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, max_q_len,
                                                    max_blocks_per_seq, max_total_len=0) -> int:
    return int(_lib.pkv_paged_attention_prefill_int4_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                                                                    max_q_len, max_blocks_per_seq, max_total_len))


def pkv_paged_attention_prefill_int4(q, k_cache, v_cache, k_scale, v_scale, block_tables, starts, cu_q, scale: float,
                                     max_q_len: int, *, max_total_len: int = 0, softcap: float = 0.0, alibi_slopes=None,
                                     key_starts=None, prefix_lens=None, out=None, workspace=None, err_flag=None,
                                     stream=None):
    """Prefill attention over 4-bit caches (as pkv_store_kvcache_int4 writes them), with the score
    rules of pkv_paged_attention_prefill_mod.  max_total_len, a bound on a sequence's positions
    (0: the tables' width), bounds the workspace."""
    nb, Hkv, bs, d = _int4_cache(k_cache, v_cache, k_scale, v_scale)
    dev = _device_of(q, k_cache, v_cache, k_scale, v_scale, block_tables, starts, cu_q, alibi_slopes, key_starts,
                     prefix_lens, out, workspace, err_flag)
    dtype, shape, tables, B = q.dtype, q.shape, block_tables.shape, starts.numel()
    if dtype not in _DTYPE:
        raise TypeError("q must be float16/bfloat16")
    if len(shape) != 3 or shape[2] != d:
        raise ValueError(f"q must be [rows, Hq, {d}]")
    _want_i32(block_tables=block_tables, starts=starts, cu_q=cu_q)
    if cu_q.numel() != B + 1 or len(tables) != 2 or tables[0] != B:
        raise ValueError("inconsistent shapes")
    rows, Hq = shape[0], shape[1]
    mod = _score_mod(softcap, alibi_slopes, key_starts, prefix_lens, Hq, rows, B)
    if out is None:
        out = _empty(shape, dtype, dev, stream)
    elif out.shape != shape or out.dtype is not dtype:
        raise ValueError("out must have the shape and type of q")
    ws = _lib.pkv_paged_attention_prefill_int4_workspace_size(B, Hq, Hkv, d, bs, max_q_len, tables[1], max_total_len)
    if ws and workspace is None:
        workspace = _empty(ws, torch.uint8, dev, stream)
    _call(dev, _lib.pkv_paged_attention_prefill_int4, *_addrs(out, q, k_cache, v_cache, k_scale, v_scale),
          block_tables.data_ptr(), tables[1], starts.data_ptr(), cu_q.data_ptr(), B, max_q_len, max_total_len, Hq, Hkv, d, bs, nb,
          scale, mod, _DTYPE[dtype], workspace.data_ptr() if ws else None,
          workspace.numel() * workspace.element_size() if ws else 0, _flag(err_flag), _raw_stream(dev, stream))
    return out


# ----------------------------------------------------------------------------- failure detection
def pkv_selftest_wait_timeout(err_flag, timeout_us: int, *, stream=None):
    """Runs the bounded pipeline wait on a barrier nothing completes: after
    `timeout_us` the kernel sets ERRBIT_TIMEOUT in `err_flag` (device int32)."""
    dev = _dev(err_flag)
    _want(err_flag, torch.int32, "err_flag")
    with torch.cuda.device(dev):
        _check(_lib.pkv_selftest_wait_timeout(_ptr(err_flag), int(timeout_us), _stream(dev, stream)))


# ----------------------------------------------------------------------------- host block allocator
class BlockAllocator:
    """Handle of a host block allocator (see pkv_allocator_* in pkv.h); the
    pool is freed with the object."""

    def __init__(self, num_blocks: int, block_size: int):
        h = ctypes.c_void_p()
        _check(_lib.pkv_allocator_create(num_blocks, block_size, ctypes.byref(h)))
        self._h, self.num_blocks, self.block_size = h, num_blocks, block_size

    def __del__(self):
        h, self._h = getattr(self, "_h", None), None
        if h:
            _lib.pkv_allocator_destroy(h)


def pkv_allocator_create(num_blocks: int, block_size: int) -> BlockAllocator:
    return BlockAllocator(num_blocks, block_size)


def pkv_allocator_add_sequence(a: BlockAllocator, seq: int, num_tokens: int, blocks=None):
    arr = None
    if blocks is not None:
        blocks = list(blocks)
        arr = (ctypes.c_int32 * max(1, len(blocks)))(*blocks)
        if len(blocks) < -(-num_tokens // a.block_size):
            raise ValueError("blocks must cover num_tokens")
    _check(_lib.pkv_allocator_add_sequence(a._h, seq, num_tokens, arr))


def pkv_allocator_fork(a: BlockAllocator, parent: int, child: int, num_tokens: int):
    _check(_lib.pkv_allocator_fork(a._h, parent, child, num_tokens))


def pkv_allocator_append(a: BlockAllocator, seq: int, num_tokens: int = 1) -> list:
    """Grows the sequence; returns the slots of its new positions."""
    arr = (ctypes.c_int32 * max(1, num_tokens))()
    _check(_lib.pkv_allocator_append(a._h, seq, num_tokens, arr))
    return list(arr[:num_tokens])


def pkv_allocator_release(a: BlockAllocator, seq: int):
    _check(_lib.pkv_allocator_release(a._h, seq))


def pkv_allocator_block_table(a: BlockAllocator, seq: int, max_blocks: int):
    """(row of max_blocks block ids padded with -1, length in tokens, blocks used)."""
    row = (ctypes.c_int32 * max(1, max_blocks))()
    n, used = ctypes.c_int64(), ctypes.c_int32()
    _check(_lib.pkv_allocator_block_table(a._h, seq, row, max_blocks, ctypes.byref(n), ctypes.byref(used)))
    return list(row[:max_blocks]), n.value, used.value


def pkv_allocator_stats(a: BlockAllocator) -> dict:
    v = [ctypes.c_int64() for _ in range(4)]
    _check(_lib.pkv_allocator_stats(a._h, *[ctypes.byref(x) for x in v]))
    return dict(zip(("free", "allocated", "referenced", "sequences"), (x.value for x in v)))


def pkv_allocator_check(a: BlockAllocator) -> int:
    return int(_lib.pkv_allocator_check(a._h))
