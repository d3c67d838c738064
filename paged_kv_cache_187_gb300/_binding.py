"""ctypes binding of libpa.so: the C ABI of include/pa.h with the same names.

Argument marshalling only.  Every function takes torch tensors (for device buffers)
or numpy arrays (for the host allocator), checks dtype / shape / device / contiguity,
derives the sizes the C call needs, and passes raw pointers.  All arithmetic happens
in the CUDA library; there is no fallback.  Importing this module on a machine
without the built library raises immediately.
"""
from __future__ import annotations

import array
import ctypes
import operator
import os

import numpy as np

from . import build as _build


class _Torch:
    """Stands for torch until a call takes something of it: the allocator and raw() need none."""

    def __getattr__(self, name):
        _with_torch()
        return getattr(torch, name)


torch = _Torch()


def _with_torch():
    """Puts torch, and what the calls take of it, in place of the stand-ins."""
    import torch as module
    global torch, _current_device, _current_stream, _is_contiguous, _device_of, _address_of
    torch, tensor = module, module.Tensor
    _current_device = getattr(module._C, "_cuda_getDevice", None)
    _current_stream = getattr(module._C, "_cuda_getCurrentRawStream", None)
    _is_contiguous, _device_of, _address_of = tensor.is_contiguous, tensor.get_device, tensor.data_ptr

_PKG = os.path.dirname(os.path.abspath(__file__))

PA_OK = 0
PA_ERR_INVALID_ARG = 1
PA_ERR_UNSUPPORTED = 2
PA_ERR_NO_BLOCKS = 3
PA_ERR_CUDA = 4
PA_ERR_WORKSPACE = 5

PA_F16 = 0
PA_BF16 = 1
PA_FP8_E4M3 = 2

PA_DEVERR_BAD_SLOT = 1
PA_DEVERR_BAD_BLOCK = 2
PA_DEVERR_BAD_LEN = 4
PA_DEVERR_TIMEOUT = 8


class PAError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"pa status {status}: {message}")
        self.status = status


class PANoBlocks(PAError):
    pass


def _load():
    path = _build.LIB
    if not os.path.exists(path):
        raise ImportError(
            f"{path} is missing: build it with paged_kv_cache_187_gb300.build.build() "
            "(nvcc for sm_103a); this package has no CPU fallback")
    lib = ctypes.CDLL(path)
    P, i32, u64, f32, sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint64, ctypes.c_float,
                            ctypes.c_size_t)
    i64 = ctypes.c_int64
    sig = {
        "pa_last_error": ([], ctypes.c_char_p),
        "pa_version": ([], i32),
        "pa_set_gqa_tensor_cores": ([i32], i32),
        "pa_set_mq_tcgen05": ([i32], i32),
        "pa_set_kernel_events": ([P, P], i32),
        "pa_selftest_wait_timeout": ([P, ctypes.c_uint32, P], i32),
        "pa_reshape_and_cache": ([P, P, P, P, P, i32, i32, i32, i32, i32, i32, P, P], i32),
        "pa_decode_v1": ([P, P, P, P, P, i32, P, i32, i32, i32, i32, i32, i32, i32, f32, i32, P, P],
                         i32),
        "pa_decode_v2_workspace_size": ([i32, i32, i32, i32, i32], sz),
        "pa_decode_v2": ([P, P, P, P, P, i32, P, i32, i32, i32, i32, i32, i32, i32, f32, i32, i32,
                          P, sz, P, P], i32),
        "pa_decode_v2_noalloc": ([P, P, P, P, P, i32, P, i32, i32, i32, i32, i32, i32, i32, f32,
                                  i32, i32, P, P], i32),
        "pa_decode_auto_plan": ([i32, i32, i32, i32, i32, i32, ctypes.POINTER(i32),
                                 ctypes.POINTER(i32)], i32),
        "pa_decode_auto_workspace_size": ([i32, i32, i32, i32, i32, i32], sz),
        "pa_decode_auto": ([P, P, P, P, P, i32, P, i32, i32, i32, i32, i32, i32, i32, f32, i32, P,
                            sz, P, P], i32),
        "pa_reshape_and_cache_fp8": ([P, P, P, P, P, i32, i32, i32, i32, i32, i32, f32, f32, P, P],
                                     i32),
        "pa_decode_fp8": ([P, P, P, P, P, i32, P, i32, i32, i32, i32, i32, i32, i32, f32, f32, f32,
                           i32, i32, i32, P, sz, P, P], i32),
        "pa_decode_mq_workspace_size": ([i32, i32, i32, i32, i32, i32, i32, i32], sz),
        "pa_decode_mq": ([P, P, P, P, P, i32, P, i32, i32, i32, i32, i32, i32, i32, i32, f32, i32,
                          i32, i32, P, sz, P, P], i32),
        "pa_decode_step": ([P, P, P, P, P, P, P, P, i32, P, i32, i32, i32, i32, i32, i32, i32, f32,
                            i32, P, sz, P, P], i32),
        "pa_decode_step_host_staging_size": ([i32, i32, i32, i32, i32], sz),
        "pa_decode_step_host": ([P, P, P, P, P, P, P, P, P, i32, i32, i32, i32, i32, i32, i32, i32,
                                 f32, i32, P, sz, P, sz, P, P], i32),
        "pa_decode_step_host_overlapped": ([P, P, P, P, P, P, P, P, P, i32, i32, i32, i32, i32, i32,
                                            i32, i32, f32, i32, P, sz, P, sz, P, P, P, P, P, P],
                                           i32),
        "pa_prefill_workspace_size": ([i32] * 6, sz),
        "pa_prefill": ([P, P, P, P, P, i32, P, P, i32, i32, i32, i32, i32, i32, i32, i32, f32, i32,
                        P, sz, P, P], i32),
        "pa_prefill_fp8": ([P, P, P, P, P, i32, P, P, i32, i32, i32, i32, i32, i32, i32, i32, f32,
                            f32, f32, i32, P, sz, P, P], i32),
        "pa_rope_and_cache": ([P, P, P, P, i64, i64, i64, P, P, P, P, i32, P, P, i32, i32, i32, i32,
                               i32, i32, i32, i32, i32, P, P], i32),
        "pa_rope_and_cache_fp8": ([P, P, P, P, i64, i64, i64, P, P, P, P, i32, P, P, i32, i32, i32,
                                   i32, i32, i32, i32, i32, i32, f32, f32, P, P], i32),
        "pa_move_blocks": ([P, P, i32, P, i32, P, i32, i32, i32, i32, i32, i32, i32, P, P], i32),
        "pa_decode_tree_workspace_size": ([i32] * 6, sz),
        "pa_decode_tree": ([P, P, P, P, P, i32, P, P, P, i32] + [i32] * 8 + [f32, i32, P, sz, P, P], i32),
        "pa_decode_tree_fp8": ([P, P, P, P, P, i32, P, P, P, i32] + [i32] * 8 +
                               [f32, f32, f32, i32, P, sz, P, P], i32),
        "pa_tree_accept": ([P, i32, P, P, P, P, P, P, i32, P, P, i32, i32, P, P], i32),
        "pa_move_tokens": ([P, P, i32, P, i32, P, P, i32, P, i32, i32, i32, i32, i32, i32, P, P], i32),
        "pa_key_bounds": ([P, P, P, P, i32, P, P, i32, i32, i32, i32, i32, i32, i32, P, P], i32),
        "pa_select_blocks_workspace_size": ([i32] * 5, sz),
        "pa_select_blocks": ([P, P, P, P, P, i32, P] + [i32] * 12 + [P, sz, P, P], i32),
        "pa_decode_sparse_workspace_size": ([i32] * 7, sz),
        "pa_decode_sparse": ([P, P, P, P, P, i32, P, P] + [i32] * 8 + [f32, i32, P, sz, P, P], i32),
        "pa_decode_sparse_fp8": ([P, P, P, P, P, i32, P, P] + [i32] * 8 +
                                 [f32, f32, f32, i32, P, sz, P, P], i32),
        "pa_alloc_shrink": ([P, i32, P, i32, ctypes.POINTER(i32)], i32),
        "pa_alloc_create": ([i32, i32, u64, ctypes.POINTER(P)], i32),
        "pa_alloc_destroy": ([P], None),
        "pa_alloc_num_free": ([P], i32),
        "pa_alloc_add_seq": ([P, i32, i32], i32),
        "pa_alloc_append": ([P, i32, ctypes.POINTER(i32)], i32),
        "pa_alloc_append_batch": ([P, P, i32, P], i32),
        "pa_alloc_free_seq": ([P, i32], i32),
        "pa_alloc_reserve_batch": ([P, P, i32, i32], i32),
        "pa_alloc_fork": ([P, i32, i32, i32], i32),
        "pa_alloc_num_pending_copies": ([P], i32),
        "pa_alloc_take_copies": ([P, P, i32, ctypes.POINTER(i32)], i32),
        "pa_alloc_refcount": ([P, i32], i32),
        "pa_copy_blocks": ([P, P, P, i32, i32, i32, i32, i32, i32, P, P], i32),
        "pa_advance_step": ([P, P, P, i32, i32, i32, i32, P, P, P, P, P], i32),
        "pa_alloc_slots": ([P, i32, i32, i32, P], i32),
        "pa_alloc_block_tables": ([P, P, i32, i32, P], i32),
        "pa_alloc_context_lens": ([P, P, i32, P], i32),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    return lib


_lib = _load()


def _check(status: int):
    if status != PA_OK:
        msg = (_lib.pa_last_error() or b"").decode()
        if status == PA_ERR_NO_BLOCKS:
            raise PANoBlocks(status, msg)
        raise PAError(status, msg)


def library_path() -> str:
    return _build.LIB


def raw():
    """The ctypes handle of libpa.so (all C symbols)."""
    return _lib


# --------------------------------------------------------------------------- helpers
def _dt(t) -> int:
    if t.dtype == torch.float16:
        return PA_F16
    if t.dtype == torch.bfloat16:
        return PA_BF16
    raise TypeError(f"unsupported dtype {t.dtype} (float16 or bfloat16)")


def _dev(t, name, dtype=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return ctypes.c_void_p(t.data_ptr())


def _opt_dev(t, name):
    if t is None:
        return None
    return _dev(t, name, torch.int32)


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


# --------------------------------------------------------------------------- kernels
def pa_reshape_and_cache(key, value, key_cache, value_cache, slot_mapping, status=None,
                         stream=None):
    """key/value [T, Hkv, D]; key_cache/value_cache [NB, Hkv, bs, D]; slot_mapping [T] int32."""
    T, Hkv, D = key.shape
    NB, Hkv2, bs, D2 = key_cache.shape
    if value.shape != key.shape or value_cache.shape != key_cache.shape or (Hkv2, D2) != (Hkv, D):
        raise ValueError("reshape_and_cache: inconsistent shapes")
    if slot_mapping.shape != (T,):
        raise ValueError("reshape_and_cache: slot_mapping must be [num_tokens]")
    dt = _dt(key)
    for t, n in ((value, "value"), (key_cache, "key_cache"), (value_cache, "value_cache")):
        if t.dtype != key.dtype:
            raise TypeError(f"{n} dtype differs from key")
    _check(_lib.pa_reshape_and_cache(
        _dev(key, "key"), _dev(value, "value"), _dev(key_cache, "key_cache"),
        _dev(value_cache, "value_cache"), _dev(slot_mapping, "slot_mapping", torch.int32),
        T, Hkv, D, bs, NB, dt, _opt_dev(status, "status"), _stream(stream)))


def _decode_common(out, query, key_cache, value_cache, block_tables, context_lens):
    S, Hq, D = query.shape
    NB, Hkv, bs, D2 = key_cache.shape
    if out.shape != query.shape or value_cache.shape != key_cache.shape or D2 != D:
        raise ValueError("decode: inconsistent shapes")
    if block_tables.dim() != 2 or block_tables.shape[0] != S or context_lens.shape != (S,):
        raise ValueError("decode: block_tables [S, max_blocks] and context_lens [S] expected")
    dt = _dt(query)
    for t, n in ((out, "out"), (key_cache, "key_cache"), (value_cache, "value_cache")):
        if t.dtype != query.dtype:
            raise TypeError(f"{n} dtype differs from query")
    ptrs = (_dev(out, "out"), _dev(query, "query"), _dev(key_cache, "key_cache"),
            _dev(value_cache, "value_cache"), _dev(block_tables, "block_tables", torch.int32),
            int(block_tables.shape[1]), _dev(context_lens, "context_lens", torch.int32))
    return ptrs, (S, Hq, Hkv, D, bs, NB), dt


def pa_decode_v1(out, query, key_cache, value_cache, block_tables, context_lens,
                 max_context_len: int, scale: float, status=None, stream=None):
    ptrs, (S, Hq, Hkv, D, bs, NB), dt = _decode_common(out, query, key_cache, value_cache,
                                                       block_tables, context_lens)
    _check(_lib.pa_decode_v1(*ptrs, S, Hq, Hkv, D, bs, NB, int(max_context_len), float(scale), dt,
                             _opt_dev(status, "status"), _stream(stream)))


def pa_decode_v2_workspace_size(num_seqs, num_q_heads, head_size, max_context_len,
                                partition_size) -> int:
    return int(_lib.pa_decode_v2_workspace_size(num_seqs, num_q_heads, head_size,
                                                max_context_len, partition_size))


def _ws(workspace):
    if workspace is None:
        return None, 0
    return _dev(workspace, "workspace"), workspace.numel() * workspace.element_size()


def pa_decode_v2(out, query, key_cache, value_cache, block_tables, context_lens,
                 max_context_len: int, scale: float, partition_size: int, workspace,
                 status=None, stream=None):
    ptrs, (S, Hq, Hkv, D, bs, NB), dt = _decode_common(out, query, key_cache, value_cache,
                                                       block_tables, context_lens)
    wp, wb = _ws(workspace)
    _check(_lib.pa_decode_v2(*ptrs, S, Hq, Hkv, D, bs, NB, int(max_context_len), float(scale), dt,
                             int(partition_size), wp, wb, _opt_dev(status, "status"),
                             _stream(stream)))


def _header_scratch_bytes() -> int:
    """PA_NOALLOC_SCRATCH_BYTES as include/pa.h defines it (the one source of the size)."""
    import re
    with open(os.path.join(os.path.dirname(_PKG), "include", "pa.h")) as f:
        m = re.search(r"#define\s+PA_NOALLOC_SCRATCH_BYTES\s+\(\(size_t\)(\d+)\s*<<\s*(\d+)\)",
                      f.read())
    if not m:
        raise ImportError("include/pa.h: PA_NOALLOC_SCRATCH_BYTES not found")
    return int(m.group(1)) << int(m.group(2))


PA_NOALLOC_SCRATCH_BYTES = _header_scratch_bytes()


def pa_decode_v2_noalloc(out, query, key_cache, value_cache, block_tables, context_lens,
                         max_context_len: int, scale: float, partition_size: int, status=None,
                         stream=None):
    """pa_decode_v2 without a workspace argument: the library's fixed device scratch is
    used instead, and nothing is allocated.  For callers that may not allocate device
    memory; calls that overlap on the GPU share that scratch and must be serialised."""
    ptrs, (S, Hq, Hkv, D, bs, NB), dt = _decode_common(out, query, key_cache, value_cache,
                                                       block_tables, context_lens)
    _check(_lib.pa_decode_v2_noalloc(*ptrs, S, Hq, Hkv, D, bs, NB, int(max_context_len),
                                     float(scale), dt, int(partition_size),
                                     _opt_dev(status, "status"), _stream(stream)))


def pa_decode_auto_plan(num_seqs, num_q_heads, num_kv_heads, head_size, block_size,
                        max_context_len):
    v, p = ctypes.c_int32(0), ctypes.c_int32(0)
    _check(_lib.pa_decode_auto_plan(num_seqs, num_q_heads, num_kv_heads, head_size, block_size,
                                    max_context_len, ctypes.byref(v), ctypes.byref(p)))
    return int(v.value), int(p.value)


def pa_decode_auto_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_size, block_size,
                                  max_context_len) -> int:
    return int(_lib.pa_decode_auto_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_size,
                                                  block_size, max_context_len))


def pa_decode_auto(out, query, key_cache, value_cache, block_tables, context_lens,
                   max_context_len: int, scale: float, workspace=None, status=None, stream=None):
    ptrs, (S, Hq, Hkv, D, bs, NB), dt = _decode_common(out, query, key_cache, value_cache,
                                                       block_tables, context_lens)
    wp, wb = _ws(workspace)
    _check(_lib.pa_decode_auto(*ptrs, S, Hq, Hkv, D, bs, NB, int(max_context_len), float(scale),
                               dt, wp, wb, _opt_dev(status, "status"), _stream(stream)))


def _u8(t, name):
    """An fp8 E4M3 pool: a uint8 (or float8_e4m3fn) CUDA tensor."""
    if t.dtype not in (torch.uint8, getattr(torch, "float8_e4m3fn", torch.uint8)):
        raise TypeError(f"{name} must be uint8 / float8_e4m3fn (fp8 E4M3 bytes), got {t.dtype}")
    return _dev(t, name)


def pa_reshape_and_cache_fp8(key, value, key_cache, value_cache, slot_mapping, k_scale: float,
                             v_scale: float, status=None, stream=None):
    """Quantising scatter: key/value [T, Hkv, D] fp16/bf16 -> fp8 E4M3 pools [NB, Hkv, bs, D]."""
    T, Hkv, D = key.shape
    NB, Hkv2, bs, D2 = key_cache.shape
    if value.shape != key.shape or value_cache.shape != key_cache.shape or (Hkv2, D2) != (Hkv, D):
        raise ValueError("reshape_and_cache_fp8: inconsistent shapes")
    if slot_mapping.shape != (T,):
        raise ValueError("reshape_and_cache_fp8: slot_mapping must be [num_tokens]")
    _check(_lib.pa_reshape_and_cache_fp8(
        _dev(key, "key"), _dev(value, "value"), _u8(key_cache, "key_cache"),
        _u8(value_cache, "value_cache"), _dev(slot_mapping, "slot_mapping", torch.int32), T, Hkv, D,
        bs, NB, _dt(key), float(k_scale), float(v_scale), _opt_dev(status, "status"),
        _stream(stream)))


_VARIANTS = {"auto": 0, "v1": 1, "v2": 2}


def pa_decode_fp8(out, query, key_cache, value_cache, block_tables, context_lens,
                  max_context_len: int, scale: float, k_scale: float, v_scale: float,
                  variant: str = "auto", partition_size: int = 0, workspace=None, status=None,
                  stream=None):
    """Paged decode over fp8 E4M3 pools; query/out fp16 or bf16 [S, Hq, D]."""
    S, Hq, D = query.shape
    NB, Hkv, bs, D2 = key_cache.shape
    if out.shape != query.shape or value_cache.shape != key_cache.shape or D2 != D:
        raise ValueError("decode_fp8: inconsistent shapes")
    if block_tables.dim() != 2 or block_tables.shape[0] != S or context_lens.shape != (S,):
        raise ValueError("decode_fp8: block_tables [S, max_blocks] and context_lens [S] expected")
    wp, wb = _ws(workspace)
    _check(_lib.pa_decode_fp8(
        _dev(out, "out"), _dev(query, "query"), _u8(key_cache, "key_cache"),
        _u8(value_cache, "value_cache"), _dev(block_tables, "block_tables", torch.int32),
        int(block_tables.shape[1]), _dev(context_lens, "context_lens", torch.int32), S, Hq, Hkv, D,
        bs, NB, int(max_context_len), float(scale), float(k_scale), float(v_scale), _dt(query),
        _VARIANTS[variant], int(partition_size or 0), wp, wb, _opt_dev(status, "status"),
        _stream(stream)))


def pa_decode_mq_workspace_size(num_seqs, q_len, num_q_heads, num_kv_heads, head_size, block_size,
                                max_context_len, partition_size=0) -> int:
    return int(_lib.pa_decode_mq_workspace_size(num_seqs, q_len, num_q_heads, num_kv_heads,
                                                head_size, block_size, max_context_len,
                                                int(partition_size or 0)))


def pa_decode_mq(out, query, key_cache, value_cache, block_tables, context_lens,
                 max_context_len: int, scale: float, variant: str = "auto", partition_size: int = 0,
                 workspace=None, status=None, stream=None):
    """Multi-query paged decode: query/out [S, q_len, Hq, D]; new token j of a sequence of
    length L attends to tokens t < L - q_len + j + 1."""
    S, QL, Hq, D = query.shape
    NB, Hkv, bs, D2 = key_cache.shape
    if out.shape != query.shape or value_cache.shape != key_cache.shape or D2 != D:
        raise ValueError("decode_mq: inconsistent shapes")
    if block_tables.dim() != 2 or block_tables.shape[0] != S or context_lens.shape != (S,):
        raise ValueError("decode_mq: block_tables [S, max_blocks] and context_lens [S] expected")
    wp, wb = _ws(workspace)
    _check(_lib.pa_decode_mq(
        _dev(out, "out"), _dev(query, "query"), _dev(key_cache, "key_cache"),
        _dev(value_cache, "value_cache"), _dev(block_tables, "block_tables", torch.int32),
        int(block_tables.shape[1]), _dev(context_lens, "context_lens", torch.int32), S, QL, Hq,
        Hkv, D, bs, NB, int(max_context_len), float(scale), _dt(query), _VARIANTS[variant],
        int(partition_size or 0), wp, wb, _opt_dev(status, "status"), _stream(stream)))


def pa_decode_step(out, query, key, value, key_cache, value_cache, slot_mapping, block_tables,
                   context_lens, max_context_len: int, scale: float, workspace=None, status=None,
                   stream=None):
    S, Hq, D = query.shape
    NB, Hkv, bs, D2 = key_cache.shape
    if key.shape != (S, Hkv, D) or value.shape != key.shape or slot_mapping.shape != (S,):
        raise ValueError("decode_step: key/value [S, Hkv, D] and slot_mapping [S] expected")
    if out.shape != query.shape or value_cache.shape != key_cache.shape or D2 != D:
        raise ValueError("decode_step: inconsistent shapes")
    dt = _dt(query)
    wp, wb = _ws(workspace)
    _check(_lib.pa_decode_step(
        _dev(out, "out"), _dev(query, "query"), _dev(key, "key"), _dev(value, "value"),
        _dev(key_cache, "key_cache"), _dev(value_cache, "value_cache"),
        _dev(slot_mapping, "slot_mapping", torch.int32),
        _dev(block_tables, "block_tables", torch.int32), int(block_tables.shape[1]),
        _dev(context_lens, "context_lens", torch.int32), S, Hq, Hkv, D, bs, NB,
        int(max_context_len), float(scale), dt, wp, wb, _opt_dev(status, "status"),
        _stream(stream)))


def pa_decode_step_host_staging_size(num_seqs, num_q_heads, num_kv_heads, head_size,
                                     max_blocks_per_seq) -> int:
    return int(_lib.pa_decode_step_host_staging_size(num_seqs, num_q_heads, num_kv_heads,
                                                     head_size, max_blocks_per_seq))


def _host(a, name, dtype=None):
    """Host buffer pointer: a CPU torch tensor or a numpy array, contiguous."""
    if hasattr(a, "is_cuda"):
        if a.is_cuda or not a.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CPU tensor")
        if dtype is not None and a.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}")
        return ctypes.c_void_p(a.data_ptr())
    arr = a
    if not arr.flags.c_contiguous:
        raise ValueError(f"{name} must be contiguous")
    return arr.ctypes.data_as(ctypes.c_void_p)


def pa_decode_step_host(out_host, query_host, key_host, value_host, slot_mapping_host,
                        block_tables_host, context_lens_host, key_cache, value_cache,
                        max_context_len: int, scale: float, staging, workspace=None,
                        status=None, stream=None):
    """One decode step from host buffers (pinned CPU tensors): H2D of the inputs,
    reshape_and_cache + decode, D2H of out, all enqueued on the stream (no wait)."""
    S, Hq, D = query_host.shape
    NB, Hkv, bs, D2 = key_cache.shape
    if key_host.shape != (S, Hkv, D) or value_host.shape != key_host.shape or D2 != D:
        raise ValueError("decode_step_host: key/value [S, Hkv, D] expected")
    if out_host.shape != query_host.shape or tuple(slot_mapping_host.shape) != (S,):
        raise ValueError("decode_step_host: out [S, Hq, D] and slot_mapping [S] expected")
    maxb = int(block_tables_host.shape[1])
    dt = _dt(key_cache)
    wp, wb = _ws(workspace)
    sp, sb = _ws(staging)
    _check(_lib.pa_decode_step_host(
        _host(out_host, "out_host"), _host(query_host, "query_host"), _host(key_host, "key_host"),
        _host(value_host, "value_host"), _host(slot_mapping_host, "slot_mapping_host"),
        _host(block_tables_host, "block_tables_host"), _host(context_lens_host, "context_lens_host"),
        _dev(key_cache, "key_cache"), _dev(value_cache, "value_cache"), maxb, S, Hq, Hkv, D, bs, NB,
        int(max_context_len), float(scale), dt, sp, sb, wp, wb, _opt_dev(status, "status"),
        _stream(stream)))


def pa_decode_step_host_overlapped(out_host, query_host, key_host, value_host,
                                   slot_mapping_host, block_tables_host, context_lens_host,
                                   key_cache, value_cache, max_context_len: int, scale: float,
                                   staging, compute_stream, h2d_stream, d2h_stream, staged_event,
                                   done_event, workspace=None, status=None):
    """pa_decode_step_host with the copies on `h2d_stream` / `d2h_stream` (see pa.h); the
    events are torch.cuda.Event objects already recorded once (so that the CUDA events
    exist)."""
    S, Hq, D = query_host.shape
    NB, Hkv, bs, D2 = key_cache.shape
    if key_host.shape != (S, Hkv, D) or value_host.shape != key_host.shape or D2 != D:
        raise ValueError("decode_step_host: key/value [S, Hkv, D] expected")
    if out_host.shape != query_host.shape or tuple(slot_mapping_host.shape) != (S,):
        raise ValueError("decode_step_host: out [S, Hq, D] and slot_mapping [S] expected")
    maxb = int(block_tables_host.shape[1])
    wp, wb = _ws(workspace)
    sp, sb = _ws(staging)
    _check(_lib.pa_decode_step_host_overlapped(
        _host(out_host, "out_host"), _host(query_host, "query_host"), _host(key_host, "key_host"),
        _host(value_host, "value_host"), _host(slot_mapping_host, "slot_mapping_host"),
        _host(block_tables_host, "block_tables_host"), _host(context_lens_host, "context_lens_host"),
        _dev(key_cache, "key_cache"), _dev(value_cache, "value_cache"), maxb, S, Hq, Hkv, D, bs, NB,
        int(max_context_len), float(scale), _dt(key_cache), sp, sb, wp, wb,
        _opt_dev(status, "status"), _stream(compute_stream), _stream(h2d_stream),
        _stream(d2h_stream), ctypes.c_void_p(staged_event.cuda_event),
        ctypes.c_void_p(done_event.cuda_event)))


def pa_set_kernel_events(start_event, stop_event):
    """torch.cuda.Event pair (already recorded once, so that the CUDA event exists) or
    (None, None) to switch the hook off."""
    if start_event is None or stop_event is None:
        _check(_lib.pa_set_kernel_events(None, None))
        return
    _check(_lib.pa_set_kernel_events(ctypes.c_void_p(start_event.cuda_event),
                                     ctypes.c_void_p(stop_event.cuda_event)))


def pa_advance_step(context_lens, slot_mapping, block_tables, block_size: int, num_blocks: int,
                    input_positions=None, input_tokens=None, sampled_token_ids=None,
                    status=None, stream=None):
    """Device-side move of every sequence to its next token (multi-step decode loop)."""
    S = int(context_lens.shape[0])
    if slot_mapping.shape != (S,) or block_tables.dim() != 2 or block_tables.shape[0] != S:
        raise ValueError("advance_step: context_lens / slot_mapping [S], block_tables [S, max]")
    def opt64(t, name):
        return None if t is None else _dev(t, name, torch.int64)
    _check(_lib.pa_advance_step(
        _dev(context_lens, "context_lens", torch.int32), _dev(slot_mapping, "slot_mapping", torch.int32),
        _dev(block_tables, "block_tables", torch.int32), int(block_tables.shape[1]), S,
        int(block_size), int(num_blocks), opt64(input_positions, "input_positions"),
        opt64(input_tokens, "input_tokens"), opt64(sampled_token_ids, "sampled_token_ids"),
        _opt_dev(status, "status"), _stream(stream)))


def pa_copy_blocks(key_cache, value_cache, block_pairs, status=None, stream=None):
    """Device copy of whole blocks old -> new for each row (old, new) of block_pairs
    (int32 [n, 2] on the device), in both pools."""
    NB, Hkv, bs, D = key_cache.shape
    if value_cache.shape != key_cache.shape or block_pairs.dim() != 2 or block_pairs.shape[1] != 2:
        raise ValueError("copy_blocks: pools [NB, Hkv, bs, D] and pairs [n, 2] expected")
    dt = PA_FP8_E4M3 if key_cache.element_size() == 1 else _dt(key_cache)
    _check(_lib.pa_copy_blocks(_dev(key_cache, "key_cache"), _dev(value_cache, "value_cache"),
                               _dev(block_pairs, "block_pairs", torch.int32),
                               int(block_pairs.shape[0]), Hkv, D, bs, NB, dt,
                               _opt_dev(status, "status"), _stream(stream)))


def pa_prefill_workspace_size(num_tokens, num_seqs, num_q_heads, num_kv_heads, head_size,
                              max_context_len) -> int:
    return int(_lib.pa_prefill_workspace_size(num_tokens, num_seqs, num_q_heads, num_kv_heads,
                                              head_size, max_context_len))


def _current_device():
    _with_torch()
    return _current_device()


def _current_stream(device):
    _with_torch()
    return _current_stream(device)


_shape_of, _dtype_of = operator.attrgetter("shape"), operator.attrgetter("dtype")
_is_contiguous, _device_of, _address_of = map(operator.methodcaller,
                                              ("is_contiguous", "get_device", "data_ptr"))


class _Call:
    """The device and stream of one call, and its tensors' addresses.  The library launches on
    the current device, so every tensor has to live there."""

    __slots__ = ("dev",)

    def __init__(self):
        self.dev = _current_device()

    def stream(self, stream):
        if stream is None:
            return _current_stream(self.dev)
        return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)

    def here(self, t, name):
        if t.get_device() != self.dev:
            if not t.is_cuda:
                raise ValueError(f"{name} must be a CUDA tensor")
            raise ValueError(f"{name} is on device {t.get_device()}, the current device is "
                             f"{self.dev}")

    def ptr(self, t, name, dtype):
        if t.get_device() != self.dev or t.dtype is not dtype or not t.is_contiguous():
            self.here(t, name)
            if t.dtype is not dtype:
                raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
            raise ValueError(f"{name} must be contiguous")
        return t.data_ptr()

    def pools(self, tensors, shape, dtype):
        """The addresses of layers' pools, which have one shape and type."""
        n = len(tensors)
        if list(map(_shape_of, tensors)).count(shape) != n:
            raise ValueError("the pools must have one shape and type")
        if (list(map(_dtype_of, tensors)).count(dtype) != n or not all(map(_is_contiguous, tensors))
                or list(map(_device_of, tensors)).count(self.dev) != n):
            for t in tensors:
                self.ptr(t, "pool", dtype)
        return array.array("Q", map(_address_of, tensors))

    def pool8(self, t, name):
        """An fp8 E4M3 pool: a uint8 or float8_e4m3fn tensor."""
        if t.dtype not in (torch.uint8, torch.float8_e4m3fn):
            raise TypeError(f"{name} must be uint8 / float8_e4m3fn (fp8 E4M3 bytes), got {t.dtype}")
        return self.ptr(t, name, t.dtype)

    def rows(self, t, name, dtype):
        """Address and token stride of a [T, H, D] tensor whose rows of one token are dense
        (a slice of a fused projection, for example)."""
        if t.get_device() != self.dev:
            self.here(t, name)
        if t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        T, H, D = t.shape
        s0, s1, s2 = t.stride()
        if (D > 1 and s2 != 1) or (H > 1 and s1 != D):
            raise ValueError(f"{name}: the rows of one token must be dense")
        return t.data_ptr(), (s0 if T > 1 else H * D)


def _prefill(fn, pool, scales, out, query, key_cache, value_cache, block_tables, context_lens,
             query_starts, max_context_len, scale, workspace, status, stream, *tree_mask):
    i32 = torch.int32
    c = _Call()
    who = "decode_tree" if tree_mask else "prefill"
    T, Hq, D = query.shape
    NB, Hkv, bs, D2 = key_cache.shape
    S = context_lens.shape[0]
    if out.shape != query.shape or value_cache.shape != key_cache.shape or D2 != D:
        raise ValueError(f"{who}: inconsistent shapes")
    if (context_lens.dim() != 1 or block_tables.dim() != 2 or block_tables.shape[0] != S
            or query_starts.dim() != 1 or query_starts.shape[0] != S + 1):
        raise ValueError(f"{who}: block_tables [S, max_blocks], context_lens [S] and "
                         "query_starts [S + 1] expected")
    tree = ()
    if tree_mask:
        mask = tree_mask[0]
        if not isinstance(mask, torch.Tensor):
            raise TypeError("decode_tree: tree_mask must be a tensor")
        if mask.dim() != 2 or mask.shape[0] != T:
            raise ValueError("decode_tree: tree_mask [T, words] expected")
        tree = (c.ptr(mask, "tree_mask", i32), mask.shape[1])
    wp, wb = None, 0
    if workspace is not None:
        wp, wb = c.ptr(workspace, "workspace", workspace.dtype), workspace.nbytes
    qt = query.dtype
    dt = _dt(query)
    if pool is None:
        k, v = c.ptr(key_cache, "key_cache", qt), c.ptr(value_cache, "value_cache", qt)
    else:
        k, v = c.pool8(key_cache, "key_cache"), c.pool8(value_cache, "value_cache")
    _check(fn(
        c.ptr(out, "out", qt), c.ptr(query, "query", qt), k, v,
        c.ptr(block_tables, "block_tables", i32), block_tables.shape[1],
        c.ptr(context_lens, "context_lens", i32), c.ptr(query_starts, "query_starts", i32), *tree, T, S, Hq,
        Hkv, D, bs, NB, max_context_len, scale, *scales, dt, wp, wb,
        None if status is None else c.ptr(status, "status", i32), c.stream(stream)))


def pa_prefill(out, query, key_cache, value_cache, block_tables, context_lens, query_starts,
               max_context_len: int, scale: float, workspace=None, status=None, stream=None):
    """Attention of a ragged chunk of new tokens over the paged cache: query/out [T, Hq, D],
    rows query_starts[s] .. query_starts[s+1]-1 belonging to sequence s's last tokens."""
    _prefill(_lib.pa_prefill, None, (), out, query, key_cache, value_cache, block_tables,
             context_lens, query_starts, int(max_context_len), float(scale), workspace, status,
             stream)


def pa_prefill_fp8(out, query, key_cache, value_cache, block_tables, context_lens, query_starts,
                   max_context_len: int, scale: float, k_scale: float, v_scale: float,
                   workspace=None, status=None, stream=None):
    """pa_prefill over fp8 E4M3 pools (uint8 or float8_e4m3fn), head_size 128."""
    _prefill(_lib.pa_prefill_fp8, True, (float(k_scale), float(v_scale)), out, query, key_cache,
             value_cache, block_tables, context_lens, query_starts, int(max_context_len),
             float(scale), workspace, status, stream)


def _rope(fn, fp8, scales, query_out, query, key, value, key_cache, value_cache, slot_mapping,
          positions, inv_freq, pair_axes, interleaved, status, stream):
    c = _Call()
    T, Hq, D = query.shape
    Hkv = key.shape[1]
    NB, Hkv2, bs, D2 = key_cache.shape
    if (key.shape != (T, Hkv, D) or value.shape != key.shape or query_out.shape != query.shape
            or value_cache.shape != key_cache.shape or (Hkv2, D2) != (Hkv, D)):
        raise ValueError("rope_and_cache: inconsistent shapes")
    if slot_mapping.shape != (T,) or positions.dim() != 2 or positions.shape[1] != T:
        raise ValueError("rope_and_cache: slot_mapping [T] and positions [axes, T] expected")
    if inv_freq.dim() != 1:
        raise ValueError("rope_and_cache: inv_freq [rot_dim / 2] expected")
    half = inv_freq.shape[0]
    axes = None
    if pair_axes is not None:
        axes = array.array("i", pair_axes)
        if len(axes) != half:
            raise ValueError("rope_and_cache: pair_axes must name one axis per pair")
    dt, qt = _dt(query), query.dtype
    qp, qs = c.rows(query, "query", qt)
    kp, ks = c.rows(key, "key", qt)
    vp, vs = c.rows(value, "value", qt)
    if fp8:
        kc, vc = c.pool8(key_cache, "key_cache"), c.pool8(value_cache, "value_cache")
    else:
        kc, vc = c.ptr(key_cache, "key_cache", qt), c.ptr(value_cache, "value_cache", qt)
    _check(fn(
        c.ptr(query_out, "query_out", qt), qp, kp, vp, qs, ks, vs, kc, vc,
        c.ptr(slot_mapping, "slot_mapping", torch.int32), c.ptr(positions, "positions", torch.int64),
        positions.shape[0], None if axes is None else axes.buffer_info()[0],
        c.ptr(inv_freq, "inv_freq", torch.float32), 2 * half, 1 if interleaved else 0, T, Hq, Hkv, D,
        bs, NB, dt, *scales, None if status is None else c.ptr(status, "status", torch.int32),
        c.stream(stream)))


def pa_rope_and_cache(query_out, query, key, value, key_cache, value_cache, slot_mapping, positions,
                      inv_freq, pair_axes=None, interleaved: bool = False, status=None, stream=None):
    """Rotary positions on query/key [T, H, D] and the K/V rows into the pools.  positions
    int64 [axes, T]; inv_freq fp32 [rot_dim / 2]; pair_axes (a sequence of ints on the
    host) names the axis of each rotated pair, needed for more than
    one axis.  query/key/value may be slices of a fused projection; query_out is dense."""
    _rope(_lib.pa_rope_and_cache, False, (), query_out, query, key, value, key_cache, value_cache,
          slot_mapping, positions, inv_freq, pair_axes, interleaved, status, stream)


def pa_rope_and_cache_fp8(query_out, query, key, value, key_cache, value_cache, slot_mapping,
                          positions, inv_freq, k_scale: float, v_scale: float, pair_axes=None,
                          interleaved: bool = False, status=None, stream=None):
    """pa_rope_and_cache into fp8 E4M3 pools (uint8 or float8_e4m3fn)."""
    _rope(_lib.pa_rope_and_cache_fp8, True, (float(k_scale), float(v_scale)), query_out, query, key,
          value, key_cache, value_cache, slot_mapping, positions, inv_freq, pair_axes, interleaved,
          status, stream)


def pa_move_blocks(key_caches, value_caches, block_pairs, block_tables=None, status=None,
                   stream=None):
    """Moves block `from` to block `to` for each row (from, to) of block_pairs (int32 [n, 2]
    on the device, ascending `from`) in every layer's pools (lists of [NB, Hkv, bs, D]
    tensors), and rewrites block_tables (int32 [rows, max_blocks] on the device)."""
    c = _Call()
    L = len(key_caches)
    if L == 0 or len(value_caches) != L:
        raise ValueError("move_blocks: key_caches and value_caches of at least one layer expected")
    if block_pairs.dim() != 2 or block_pairs.shape[1] != 2:
        raise ValueError("move_blocks: pairs [n, 2] expected")
    k0 = key_caches[0]
    NB, Hkv, bs, D = shape = k0.shape
    pt = k0.dtype
    dt = PA_FP8_E4M3 if k0.element_size() == 1 else _dt(k0)
    if dt == PA_FP8_E4M3:
        c.pool8(k0, "pool")
    pools = []
    for t in (*key_caches, *value_caches):
        if t.shape != shape:
            raise ValueError("move_blocks: the pools must have one shape and type")
        pools.append(c.ptr(t, "pool", pt))
    pools = np.array(pools, dtype=np.uint64)
    rows, width, tables = 0, 1, None
    if block_tables is not None:
        if block_tables.dim() != 2:
            raise ValueError("move_blocks: block_tables [rows, max_blocks] expected")
        rows, width = block_tables.shape
        tables = c.ptr(block_tables, "block_tables", torch.int32)
    base = pools.ctypes.data
    _check(_lib.pa_move_blocks(
        base, base + 8 * L, L, c.ptr(block_pairs, "block_pairs", torch.int32), block_pairs.shape[0],
        tables, rows, width, Hkv, D, bs, NB, dt,
        None if status is None else c.ptr(status, "status", torch.int32), c.stream(stream)))


def pa_decode_tree_workspace_size(num_tokens, num_seqs, num_q_heads, num_kv_heads, head_size,
                                  max_context_len) -> int:
    return int(_lib.pa_decode_tree_workspace_size(num_tokens, num_seqs, num_q_heads, num_kv_heads,
                                                  head_size, max_context_len))


def pa_decode_tree(out, query, key_cache, value_cache, block_tables, context_lens, query_starts,
                   tree_mask, max_context_len: int, scale: float, workspace=None, status=None,
                   stream=None):
    """pa_prefill for new tokens that form a tree: tree_mask int32 [T, words], bit i % 32 of word
    i / 32 of a token's row set if the token sees new token i of its sequence."""
    _prefill(_lib.pa_decode_tree, None, (), out, query, key_cache, value_cache, block_tables,
             context_lens, query_starts, int(max_context_len), float(scale), workspace, status,
             stream, tree_mask)


def pa_decode_tree_fp8(out, query, key_cache, value_cache, block_tables, context_lens, query_starts,
                       tree_mask, max_context_len: int, scale: float, k_scale: float, v_scale: float,
                       workspace=None, status=None, stream=None):
    """pa_decode_tree over fp8 E4M3 pools (uint8 or float8_e4m3fn), head_size 128."""
    _prefill(_lib.pa_decode_tree_fp8, True, (float(k_scale), float(v_scale)), out, query, key_cache,
             value_cache, block_tables, context_lens, query_starts, int(max_context_len),
             float(scale), workspace, status, stream, tree_mask)


def pa_tree_accept(accepted, num_accepted, next_tokens, new_lens, draft_tokens, target_tokens,
                   tree_mask, query_starts, context_lens, status=None, stream=None):
    """The path of each tree that the model's choices accept: accepted int32 [S, max_accepted],
    num_accepted int32 [S], next_tokens int64 [S], new_lens int32 [S] (may be context_lens), from
    draft_tokens / target_tokens int64 [T] and tree_mask int32 [T, words]."""
    i32, i64 = torch.int32, torch.int64
    c = _Call()
    T, S = draft_tokens.shape[0], context_lens.shape[0]
    if (accepted.dim() != 2 or accepted.shape[0] != S or num_accepted.shape != (S,)
            or next_tokens.shape != (S,) or new_lens.shape != (S,) or context_lens.dim() != 1
            or query_starts.shape != (S + 1,)):
        raise ValueError("tree_accept: accepted [S, max_accepted]; num_accepted, next_tokens, "
                         "new_lens, context_lens [S] and query_starts [S + 1] expected")
    if draft_tokens.dim() != 1 or target_tokens.shape != (T,) or tree_mask.dim() != 2 or tree_mask.shape[0] != T:
        raise ValueError("tree_accept: draft_tokens, target_tokens [T] and tree_mask [T, words] expected")
    _check(_lib.pa_tree_accept(
        c.ptr(accepted, "accepted", i32), accepted.shape[1], c.ptr(num_accepted, "num_accepted", i32),
        c.ptr(next_tokens, "next_tokens", i64), c.ptr(new_lens, "new_lens", i32),
        c.ptr(draft_tokens, "draft_tokens", i64), c.ptr(target_tokens, "target_tokens", i64),
        c.ptr(tree_mask, "tree_mask", i32), tree_mask.shape[1], c.ptr(query_starts, "query_starts", i32),
        c.ptr(context_lens, "context_lens", i32), T, S,
        None if status is None else c.ptr(status, "status", i32), c.stream(stream)))


def pa_move_tokens(key_caches, value_caches, block_tables, new_lens, accepted, num_accepted,
                   status=None, stream=None):
    """Moves the rows of the accepted tokens together in every layer's pools (lists of
    [NB, Hkv, bs, D] tensors): position b + accepted[s][j] to b + j, b = new_lens[s] -
    num_accepted[s]."""
    i32 = torch.int32
    c = _Call()
    L = len(key_caches)
    if L == 0 or len(value_caches) != L:
        raise ValueError("move_tokens: key_caches and value_caches of at least one layer expected")
    k0 = key_caches[0]
    NB, Hkv, bs, D = shape = k0.shape
    S = new_lens.shape[0]
    if (block_tables.dim() != 2 or block_tables.shape[0] != S or new_lens.dim() != 1
            or accepted.dim() != 2 or accepted.shape[0] != S or num_accepted.shape != (S,)):
        raise ValueError("move_tokens: block_tables [S, max_blocks], new_lens and num_accepted [S], "
                         "accepted [S, max_accepted] expected")
    pt = k0.dtype
    dt = PA_FP8_E4M3 if k0.element_size() == 1 else _dt(k0)
    if dt == PA_FP8_E4M3:
        c.pool8(k0, "pool")
    pools = c.pools((*key_caches, *value_caches), shape, pt)
    base = pools.buffer_info()[0]
    _check(_lib.pa_move_tokens(
        base, base + 8 * L, L, c.ptr(block_tables, "block_tables", i32), block_tables.shape[1],
        c.ptr(new_lens, "new_lens", i32), c.ptr(accepted, "accepted", i32), accepted.shape[1],
        c.ptr(num_accepted, "num_accepted", i32), S, Hkv, D, bs, NB, dt,
        None if status is None else c.ptr(status, "status", i32), c.stream(stream)))


def pa_key_bounds(bounds, bound_steps, key_cache, block_tables, context_lens, max_new_tokens: int,
                  query_starts=None, status=None, stream=None):
    """Bounds of the keys of the blocks that hold each sequence's last tokens: max_new_tokens each,
    or query_starts[s + 1] - query_starts[s] of them.  bounds int8 [NB, Hkv, 2, D] (largest, then
    smallest), bound_steps fp32 [NB, Hkv]."""
    i32 = torch.int32
    c = _Call()
    NB, Hkv, bs, D = key_cache.shape
    S = context_lens.shape[0]
    if bounds.shape != (NB, Hkv, 2, D) or bound_steps.shape != (NB, Hkv):
        raise ValueError("key_bounds: bounds [NB, Hkv, 2, D] and bound_steps [NB, Hkv] expected")
    if (context_lens.dim() != 1 or block_tables.dim() != 2 or block_tables.shape[0] != S
            or (query_starts is not None and query_starts.shape != (S + 1,))):
        raise ValueError("key_bounds: block_tables [S, max_blocks], context_lens [S] and "
                         "query_starts [S + 1] expected")
    if key_cache.element_size() == 1:
        dt, k = PA_FP8_E4M3, c.pool8(key_cache, "key_cache")
    else:
        dt, k = _dt(key_cache), c.ptr(key_cache, "key_cache", key_cache.dtype)
    _check(_lib.pa_key_bounds(
        c.ptr(bounds, "bounds", torch.int8), c.ptr(bound_steps, "bound_steps", torch.float32), k,
        c.ptr(block_tables, "block_tables", i32), block_tables.shape[1],
        c.ptr(context_lens, "context_lens", i32),
        None if query_starts is None else c.ptr(query_starts, "query_starts", i32),
        int(max_new_tokens), S, Hkv, D, bs, NB, dt,
        None if status is None else c.ptr(status, "status", i32), c.stream(stream)))


def pa_select_blocks_workspace_size(num_seqs, q_len, num_kv_heads, block_size, max_context_len) -> int:
    return int(_lib.pa_select_blocks_workspace_size(num_seqs, q_len, num_kv_heads, block_size,
                                                    max_context_len))


def _rows4(t, name):
    """Shape of query tokens [S, q_len, ..]; [S, ..] is one query token each."""
    if t.dim() == 4:
        return tuple(t.shape)
    if t.dim() != 3:
        raise ValueError(f"{name} must be [S, q_len, heads, ..] or [S, heads, ..]")
    return t.shape[0], 1, t.shape[1], t.shape[2]


def pa_select_blocks(selected, query, bounds, bound_steps, block_tables, context_lens, block_size: int,
                     max_context_len: int, num_first: int, num_last: int, workspace=None, status=None,
                     stream=None):
    """The blocks that each query token and kv head reads: selected int32 [S, q_len, Hkv, n] (or
    [S, Hkv, n]), ascending, then -1; query [S, q_len, Hq, D] (or [S, Hq, D])."""
    i32 = torch.int32
    c = _Call()
    S, QL, Hq, D = _rows4(query, "query")
    S2, QL2, Hkv, n = _rows4(selected, "selected")
    NB = bounds.shape[0]
    if (S2, QL2) != (S, QL) or bounds.shape != (NB, Hkv, 2, D) or bound_steps.shape != (NB, Hkv):
        raise ValueError("select_blocks: inconsistent shapes")
    if context_lens.shape != (S,) or block_tables.dim() != 2 or block_tables.shape[0] != S:
        raise ValueError("select_blocks: block_tables [S, max_blocks] and context_lens [S] expected")
    wp, wb = None, 0
    if workspace is not None:
        wp, wb = c.ptr(workspace, "workspace", workspace.dtype), workspace.nbytes
    _check(_lib.pa_select_blocks(
        c.ptr(selected, "selected", i32), c.ptr(query, "query", query.dtype),
        c.ptr(bounds, "bounds", torch.int8), c.ptr(bound_steps, "bound_steps", torch.float32),
        c.ptr(block_tables, "block_tables", i32), block_tables.shape[1],
        c.ptr(context_lens, "context_lens", i32), S, QL, Hq, Hkv, D, int(block_size), NB,
        int(max_context_len), n, int(num_first), int(num_last), _dt(query), wp, wb,
        None if status is None else c.ptr(status, "status", i32), c.stream(stream)))


def pa_decode_sparse_workspace_size(num_seqs, q_len, num_q_heads, num_kv_heads, head_size, block_size,
                                    num_selected) -> int:
    return int(_lib.pa_decode_sparse_workspace_size(num_seqs, q_len, num_q_heads, num_kv_heads,
                                                    head_size, block_size, num_selected))


def _sparse(fn, pool, scales, out, query, key_cache, value_cache, block_tables, context_lens, selected,
            scale, workspace, status, stream):
    i32 = torch.int32
    c = _Call()
    S, QL, Hq, D = _rows4(query, "query")
    S2, QL2, Hkv, n = _rows4(selected, "selected")
    NB, Hkv2, bs, D2 = key_cache.shape
    if (out.shape != query.shape or value_cache.shape != key_cache.shape
            or (S2, QL2, Hkv2, D2) != (S, QL, Hkv, D)):
        raise ValueError("decode_sparse: inconsistent shapes")
    if context_lens.shape != (S,) or block_tables.dim() != 2 or block_tables.shape[0] != S:
        raise ValueError("decode_sparse: block_tables [S, max_blocks] and context_lens [S] expected")
    wp, wb = None, 0
    if workspace is not None:
        wp, wb = c.ptr(workspace, "workspace", workspace.dtype), workspace.nbytes
    qt = query.dtype
    dt = _dt(query)
    if pool is None:
        k, v = c.ptr(key_cache, "key_cache", qt), c.ptr(value_cache, "value_cache", qt)
    else:
        k, v = c.pool8(key_cache, "key_cache"), c.pool8(value_cache, "value_cache")
    _check(fn(
        c.ptr(out, "out", qt), c.ptr(query, "query", qt), k, v,
        c.ptr(block_tables, "block_tables", i32), block_tables.shape[1],
        c.ptr(context_lens, "context_lens", i32), c.ptr(selected, "selected", i32), n, S, QL, Hq, Hkv, D,
        bs, NB, scale, *scales, dt, wp, wb,
        None if status is None else c.ptr(status, "status", i32), c.stream(stream)))


def pa_decode_sparse(out, query, key_cache, value_cache, block_tables, context_lens, selected,
                     scale: float, workspace=None, status=None, stream=None):
    """Attention of query tokens [S, q_len, Hq, D] (or [S, Hq, D]) over the blocks that selected
    int32 [S, q_len, Hkv, n] (or [S, Hkv, n]) names."""
    _sparse(_lib.pa_decode_sparse, None, (), out, query, key_cache, value_cache, block_tables,
            context_lens, selected, float(scale), workspace, status, stream)


def pa_decode_sparse_fp8(out, query, key_cache, value_cache, block_tables, context_lens, selected,
                         scale: float, k_scale: float, v_scale: float, workspace=None, status=None,
                         stream=None):
    """pa_decode_sparse over fp8 E4M3 pools (uint8 or float8_e4m3fn), head_size 128."""
    _sparse(_lib.pa_decode_sparse_fp8, True, (float(k_scale), float(v_scale)), out, query, key_cache,
            value_cache, block_tables, context_lens, selected, float(scale), workspace, status, stream)


def pa_selftest_wait_timeout(status, limit_us: int, stream=None):
    """Runs the bounded-wait self-test kernel; sets PA_DEVERR_TIMEOUT in `status`."""
    _check(_lib.pa_selftest_wait_timeout(_dev(status, "status", torch.int32), int(limit_us),
                                         _stream(stream)))


def pa_set_gqa_tensor_cores(enable: bool):
    """Process-wide: True (default) decodes grouped-query heads and fp8 caches on the
    tensor cores, False on the CUDA cores (groups above 8 stay on the tensor cores)."""
    _check(_lib.pa_set_gqa_tensor_cores(1 if enable else 0))


def pa_set_mq_tcgen05(enable: bool):
    """Process-wide: True (default) lets multi-query decode with many rows per kv head
    use the tcgen05 kernel, False keeps it on the mma.sync kernel."""
    _check(_lib.pa_set_mq_tcgen05(1 if enable else 0))


# --------------------------------------------------------------------------- allocator
def _np_i32(a):
    return np.ascontiguousarray(a, dtype=np.int32)


def _nptr(a):
    return a.ctypes.data_as(ctypes.c_void_p)


class PagedAllocator:
    """Host block allocator (pa_alloc_* calls): builds block tables and slot mappings."""

    def __init__(self, num_blocks: int, block_size: int, seed: int):
        h = ctypes.c_void_p()
        _check(_lib.pa_alloc_create(int(num_blocks), int(block_size),
                                    int(seed) & (2**64 - 1), ctypes.byref(h)))
        self._h = h
        self.num_blocks = int(num_blocks)
        self.block_size = int(block_size)

    def close(self):
        if self._h:
            _lib.pa_alloc_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def num_free(self) -> int:
        return int(_lib.pa_alloc_num_free(self._h))

    def pa_alloc_add_seq(self, seq_id: int, num_tokens: int):
        _check(_lib.pa_alloc_add_seq(self._h, int(seq_id), int(num_tokens)))

    def pa_alloc_append(self, seq_id: int) -> int:
        s = ctypes.c_int32(0)
        _check(_lib.pa_alloc_append(self._h, int(seq_id), ctypes.byref(s)))
        return int(s.value)

    @staticmethod
    def _out(out, shape):
        if out is None:
            return np.empty(shape, dtype=np.int32)
        if out.dtype != np.int32 or out.shape != tuple(shape) or not out.flags.c_contiguous:
            raise ValueError(f"out must be a contiguous int32 array of shape {tuple(shape)}")
        return out

    def pa_alloc_append_batch(self, seq_ids, out=None) -> np.ndarray:
        ids = _np_i32(seq_ids)
        out = self._out(out, (ids.size,))
        _check(_lib.pa_alloc_append_batch(self._h, _nptr(ids), ids.size, _nptr(out)))
        return out

    def pa_alloc_reserve_batch(self, seq_ids, extra_tokens: int):
        ids = _np_i32(seq_ids)
        _check(_lib.pa_alloc_reserve_batch(self._h, _nptr(ids), ids.size, int(extra_tokens)))

    def pa_alloc_fork(self, src_seq: int, dst_seq: int, num_tokens: int):
        _check(_lib.pa_alloc_fork(self._h, int(src_seq), int(dst_seq), int(num_tokens)))

    def pa_alloc_take_copies(self) -> np.ndarray:
        """Pending copy-on-write pairs [n, 2] (old, new), cleared."""
        n = int(_lib.pa_alloc_num_pending_copies(self._h))
        out = np.zeros((max(n, 1), 2), dtype=np.int32)
        got = ctypes.c_int32(0)
        _check(_lib.pa_alloc_take_copies(self._h, _nptr(out), n, ctypes.byref(got)))
        return out[:got.value]

    def pa_alloc_refcount(self, block: int) -> int:
        return int(_lib.pa_alloc_refcount(self._h, int(block)))

    def pa_alloc_free_seq(self, seq_id: int):
        _check(_lib.pa_alloc_free_seq(self._h, int(seq_id)))

    def pa_alloc_shrink(self, num_blocks: int) -> np.ndarray:
        """Shrinks the pool to num_blocks blocks; the moved blocks' pairs [n, 2] (from, to)."""
        room = max(self.num_blocks - int(num_blocks), 0)
        out = np.zeros((max(room, 1), 2), dtype=np.int32)
        got = ctypes.c_int32(0)
        _check(_lib.pa_alloc_shrink(self._h, int(num_blocks), _nptr(out), room, ctypes.byref(got)))
        self.num_blocks = int(num_blocks)
        return out[:got.value]

    def pa_alloc_slots(self, seq_id: int, start: int, n: int) -> np.ndarray:
        out = np.empty(int(n), dtype=np.int32)
        _check(_lib.pa_alloc_slots(self._h, int(seq_id), int(start), int(n), _nptr(out)))
        return out

    def pa_alloc_block_tables(self, seq_ids, max_blocks_per_seq: int, out=None) -> np.ndarray:
        ids = _np_i32(seq_ids)
        out = self._out(out, (ids.size, int(max_blocks_per_seq)))
        _check(_lib.pa_alloc_block_tables(self._h, _nptr(ids), ids.size, int(max_blocks_per_seq),
                                          _nptr(out)))
        return out

    def pa_alloc_context_lens(self, seq_ids, out=None) -> np.ndarray:
        ids = _np_i32(seq_ids)
        out = self._out(out, (ids.size,))
        _check(_lib.pa_alloc_context_lens(self._h, _nptr(ids), ids.size, _nptr(out)))
        return out
