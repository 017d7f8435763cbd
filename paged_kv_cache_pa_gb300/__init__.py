"""GB300-native paged KV cache decode path.

Python binding of ``libpa_gb300.so`` (the C ABI declared in ``include/pa.h``)
with the same operation names.  This module only marshals arguments (device
pointers of torch tensors, sizes, the current CUDA stream); every step of the
path runs in the library's CUDA kernels.  There is no CPU fallback: calling an
operation without the built library, or with tensors that are not on a CUDA
device, or not on the current one, raises.

    cache_write(key, value, k_cache, v_cache, slot_mapping)
    decode_attention(query, k_cache, v_cache, block_tables, context_lens,
                     max_context_len, scale, out=None, ...)
    copy_blocks(k_caches, v_caches, block_pairs)
    swap_blocks(dst_k_caches, dst_v_caches, src_k_caches, src_v_caches, block_pairs)
    prefill_attention(query, k_cache, v_cache, block_tables, query_start_loc,
                      context_lens, max_query_len, max_context_len, scale, ...)

A cache that stays within a budget:

    rotary_cache_write(query, key, value, positions, rotary, k_cache, v_cache,
                       slot_mapping, ...)
    decode_attention_scored(query, k_cache, v_cache, block_tables, context_lens,
                            max_context_len, scale, scores, ...)
    prefill_scores(query, lse, k_cache, block_tables, query_start_loc, context_lens,
                   max_query_len, max_context_len, scale, scores, ...)
    evict_tokens(k_caches, v_caches, scores, block_tables, context_lens, keep_lens,
                 max_context_len, max_keep_len, num_sink, num_recent, ...)

Pools are [num_blocks][num_kv_heads][block_size][head_dim]; the block size
is read from their third dimension: 16 goes to the plain entry points, other
supported sizes (powers of two from 8 to 256) to the ``*_ex`` ones.

A call runs on ``stream`` (default: the current stream).  Tensors that it makes
belong to that stream, as if made under ``torch.cuda.stream(stream)``: before
another stream uses one that the call returns, it has to wait for the call, as
for any tensor.  Tensors that the caller passes are the caller's to keep alive
and to order.

Build the library with ``python -m paged_kv_cache_pa_gb300.build``.
"""
from __future__ import annotations

import array
import ctypes
import os
import threading
from typing import Optional, Sequence

__all__ = ["cache_write", "decode_attention", "decode_attention_contiguous",
           "decode_workspace_size", "decode_partition_tokens", "decode_kernel_launches",
           "copy_blocks",
           "status_string", "PaError", "library_path", "load_library", "BLOCK_SIZE",
           "ERRBIT_BLOCK_OOB", "ERRBIT_SLOT_OOB", "ERRBIT_CONTEXT_LEN", "ERRBIT_TIMEOUT",
           "ERRBIT_INTERNAL",
           "MAX_LAYERS", "BLOCK_SIZES", "swap_blocks", "prefill_attention",
           "Rotary", "rotary_cache_write", "decode_attention_scored",
           "decode_scored_workspace_size", "prefill_scores", "prefill_scores_workspace_size",
           "evict_tokens", "evict_workspace_size", "MAX_ROTARY_PAIRS"]

BLOCK_SIZE = 16
BLOCK_SIZES = (8, 16, 32, 64, 128, 256)
MAX_LAYERS = 128
MAX_ROTARY_PAIRS = 128
PA_F16, PA_BF16, PA_F32 = 0, 1, 2
ERRBIT_BLOCK_OOB, ERRBIT_SLOT_OOB, ERRBIT_CONTEXT_LEN, ERRBIT_TIMEOUT = 1, 2, 4, 8
ERRBIT_INTERNAL = 16  # PA_DEBUG builds only

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "libpa_gb300.so")
_lib = None
_lock = threading.Lock()

# entry point -> (restype, argtypes)
_P, _I, _U64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_uint64
_I64 = ctypes.c_int64
_SIGNATURES = {
    "pa_cache_write": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P]),
    "pa_cache_write_ex": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P]),
    "pa_rotary_init": (_I, [_P, _P, _P, _I, _I, ctypes.c_float]),
    "pa_rotary_cache_write": (_I, [_P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _P, _P, _P, _P,
                                   _I, _I, _I, _I, _I, _I, _I, _P, _P]),
    "pa_decode_workspace_size": (ctypes.c_size_t, [_I, _I, _I, _I, _I]),
    "pa_decode_partition_tokens": (_I, [_I, _I, _I]),
    "pa_decode_kernel_launches": (_I, [_I, _I, _I, _I, _I]),
    "pa_decode_attention": (_I, [_P, _I, _P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _I,
                                 ctypes.c_float, _I, _P, ctypes.c_size_t, _P, _P]),
    "pa_decode_attention_ex": (_I, [_P, _I, _P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _I,
                                    _I, ctypes.c_float, _I, _P, ctypes.c_size_t, _P, _P]),
    "pa_decode_attention_contiguous": (_I, [_P, _I, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I,
                                            ctypes.c_float, _I, _P, ctypes.c_size_t, _P, _P]),
    "pa_decode_scored_workspace_size": (ctypes.c_size_t, [_I, _I, _I, _I, _I]),
    "pa_decode_attention_scored": (_I, [_P, _I, _P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _I,
                                        _I, ctypes.c_float, _I, _P, _I64, _P, ctypes.c_size_t,
                                        _P, _P]),
    "pa_copy_blocks": (_I, [_P, _P, _I, _P, _I, _I, _I, _I, _I, _P, _P]),
    "pa_copy_blocks_ex": (_I, [_P, _P, _I, _P, _I, _I, _I, _I, _I, _I, _P, _P]),
    "pa_prefill_attention": (_I, [_P, _I, _P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _I,
                                  _I, _I, _I, ctypes.c_float, _I, _P, ctypes.c_size_t, _P, _P]),
    "pa_prefill_attention_lse": (_I, [_P, _I, _P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I,
                                      _I, _I, _I, _I, ctypes.c_float, _I, _P, _P,
                                      ctypes.c_size_t, _P, _P]),
    "pa_prefill_scores": (_I, [_P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I,
                               ctypes.c_float, _I, _P, _I64, _P, ctypes.c_size_t, _P, _P]),
    "pa_prefill_scores_workspace_size": (ctypes.c_size_t, [_I, _I, _I, _I, _I, _I]),
    "pa_prefill_workspace_size": (ctypes.c_size_t, [_I, _I, _I, _I, _I]),
    "pa_swap_blocks": (_I, [_P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _I, _I, _P, _P]),
    "pa_evict_workspace_size": (ctypes.c_size_t, [_I, _I, _I, _I, _I]),
    "pa_evict_tokens": (_I, [_P, _P, _I, _P, _I64, _P, _I64, _P, _I64, _P, _I, _P, _I, _P, _P,
                             _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _I, _P, ctypes.c_size_t,
                             _P, _P]),
    "pa_status_string": (ctypes.c_char_p, [_I]),
}


class PaError(RuntimeError):
    def __init__(self, status: int, op: str):
        self.status = status
        super().__init__(f"{op}: {status_string(status)} ({status})")


def library_path() -> str:
    return _LIB_PATH


def load_library() -> ctypes.CDLL:
    """Load libpa_gb300.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(_LIB_PATH):
                raise RuntimeError(
                    f"{_LIB_PATH} is missing: build it with "
                    "`python -m paged_kv_cache_pa_gb300.build` (there is no fallback path)")
            lib = ctypes.CDLL(_LIB_PATH)
            for name, (res, args) in _SIGNATURES.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            _lib = lib
    return _lib


def status_string(status: int) -> str:
    return load_library().pa_status_string(int(status)).decode()


def _check(status: int, op: str) -> None:
    if status != 0:
        raise PaError(status, op)


_torch_module = None


def _torch():
    """torch, imported with the first call (an import statement in every call
    costs more than this)."""
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


_DTYPE_CODES = {}


def _dtype_code(dt) -> int:
    if not _DTYPE_CODES:
        torch = _torch()
        _DTYPE_CODES.update({torch.float16: PA_F16, torch.bfloat16: PA_BF16,
                             torch.float32: PA_F32})
    code = _DTYPE_CODES.get(dt)
    if code is None:
        raise TypeError(f"unsupported dtype {dt}")
    return code


def _dev(t, name):
    if t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name} must be a CUDA tensor" if not t.is_cuda
                     else f"{name} must be contiguous")


_several_devices = None


def _stream_ptr(stream, t) -> int:
    """Handle of ``stream``, or of the current stream; t: a CUDA tensor of the
    call, or None if it has none."""
    global _several_devices
    torch = _torch()
    if _several_devices is None:
        _several_devices = torch.cuda.device_count() > 1
    if _several_devices and t is not None and t.get_device() != torch._C._cuda_getDevice():
        # (a launch goes to the current device, whatever its pointers say)
        raise ValueError(f"the tensors are on {t.device}, which is not the current device")
    if stream is None:
        # without making a Stream object
        return torch._C._cuda_getCurrentRawStream(
            torch._C._cuda_getDevice() if t is None else t.get_device())
    return int(stream.cuda_stream)


def _empty(stream, shape, dtype, device, returned=False):
    """A new tensor for a call that runs on ``stream``.  Its memory comes from
    that stream's share of the allocator, so that neither what other streams
    still do with memory they have given back, nor what they are given once
    this tensor is dropped, meets the call's kernels.  returned: the caller
    gets it, and may drop it while the current stream still uses it."""
    torch = _torch()
    if stream is None or int(stream.cuda_stream) == torch._C._cuda_getCurrentRawStream(device.index):
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if returned:
        t.record_stream(torch.cuda.current_stream(device))
    return t


def _workspace(stream, nbytes, device):
    torch = _torch()
    return _empty(stream, max(nbytes, 256), torch.uint8, device)


def _opt_ptr(t, name):
    return None if t is None else _dev(t, name)


def cache_write(key, value, k_cache, v_cache, slot_mapping, error_word=None,
                stream=None) -> None:
    """Write key[t] / value[t] ([T][Hkv][D]) into pool slot slot_mapping[t]
    (int64; < 0 skips).  Pools: [num_blocks][Hkv][block_size][D]."""
    torch = _torch()
    if slot_mapping.dtype != torch.int64:
        raise TypeError("slot_mapping must be int64")
    nb, hkv, bs, d = k_cache.shape
    if tuple(key.shape[1:]) != (hkv, d) or key.shape != value.shape:
        raise ValueError("shape mismatch between key/value and the pools")
    if v_cache.shape != k_cache.shape or k_cache.dtype != key.dtype or v_cache.dtype != key.dtype:
        raise ValueError("pools must match each other and the key dtype")
    args = (_dev(key, "key"), _dev(value, "value"), _dev(k_cache, "k_cache"),
            _dev(v_cache, "v_cache"), _dev(slot_mapping, "slot_mapping"), key.shape[0], nb)
    tail = (hkv, d, _dtype_code(key.dtype), _opt_ptr(error_word, "error_word"),
            _stream_ptr(stream, key))
    lib = load_library()
    if bs == BLOCK_SIZE:
        _check(lib.pa_cache_write(*args, *tail), "pa_cache_write")
    else:
        _check(lib.pa_cache_write_ex(*args, bs, *tail), "pa_cache_write_ex")


class _RotaryStruct(ctypes.Structure):
    """pa_rotary_t."""
    _fields_ = [("rotary_dim", ctypes.c_int32), ("num_axes", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("scale", ctypes.c_float),
                ("turns", ctypes.c_uint64 * MAX_ROTARY_PAIRS),
                ("axis", ctypes.c_uint8 * MAX_ROTARY_PAIRS)]


class Rotary:
    """Rotary frequencies for rotary_cache_write, made once and kept.

    inv_freq: radians per position of each pair (a multiple of 8 pairs, at
    most 128), scaled variants their scaled values; axes: the position axis of
    each pair (all 0 when not given), e.g. ``[0] * 16 + [1] * 24 + [2] * 24``
    for time, height and width; interleaved: pairs are neighbouring elements
    instead of the two halves of the turned part; scale: factor on the turned
    elements."""

    def __init__(self, inv_freq: Sequence[float], axes: Optional[Sequence[int]] = None,
                 interleaved: bool = False, scale: float = 1.0):
        freqs = [float(f) for f in inv_freq]
        n = len(freqs)
        if axes is not None and len(axes) != n:
            raise ValueError("axes must name one axis per frequency")
        ax = None if axes is None else (ctypes.c_int32 * n)(*[int(a) for a in axes])
        self._struct = _RotaryStruct()
        self._ptr = ctypes.addressof(self._struct)
        _check(load_library().pa_rotary_init(
            self._ptr, ctypes.cast((ctypes.c_double * n)(*freqs), _P),
            None if ax is None else ctypes.cast(ax, _P), n, int(bool(interleaved)),
            float(scale)), "pa_rotary_init")

    # a copy has frequencies, and their address, of its own
    def __getstate__(self):
        return bytes(self._struct)

    def __setstate__(self, state):
        self._struct = _RotaryStruct.from_buffer_copy(state)
        self._ptr = ctypes.addressof(self._struct)

    @property
    def rotary_dim(self) -> int:
        return self._struct.rotary_dim

    @property
    def num_axes(self) -> int:
        return self._struct.num_axes


def _rows(t, name, row):
    """Pointer and token stride (elements) of [T][heads][D], row = heads * D,
    whose heads are dense and whose tokens may be apart (a slice of a
    projection's rows)."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.is_contiguous():
        return t.data_ptr(), row
    n, h, d = t.shape
    token, head, element = t.stride()
    if element != 1 or (h > 1 and head != d):
        raise ValueError(f"{name} must have dense heads")
    return t.data_ptr(), (token if n > 1 else row)


def rotary_cache_write(query, key, value, positions, rotary: Rotary, k_cache, v_cache,
                       slot_mapping, query_out=None, error_word=None, stream=None):
    """Turn query [T][H][D] and key [T][Hkv][D] by positions (int64
    [axes][T], or [T] for one axis) and write key and value [T][Hkv][D] into
    pool slot slot_mapping[t] (int64; < 0 skips key and value).  Token strides
    are free (slices of one projection's rows).  Returns the turned query:
    ``query_out``, ``query`` itself for an update in place, or a new dense
    tensor."""
    torch = _torch()
    nb, hkv, bs, d = k_cache.shape
    T, H, D = query.shape
    new, dt = (T, hkv, d), query.dtype
    if key.shape != new or value.shape != new or D != d:
        raise ValueError("shape mismatch between query/key/value and the pools")
    if v_cache.shape != (nb, hkv, bs, d) or not (
            dt == key.dtype == value.dtype == k_cache.dtype == v_cache.dtype):
        raise ValueError("pools, query, key and value must have one dtype, the pools one shape")
    if slot_mapping.dtype != torch.int64 or positions.dtype != torch.int64:
        raise TypeError("slot_mapping and positions must be int64")
    if slot_mapping.shape != (T,):
        raise ValueError("slot_mapping must be [T]")
    if positions.shape[-1:] != (T,) or positions.dim() > 2 or \
            (positions.shape[0] if positions.dim() == 2 else 1) < rotary.num_axes:
        raise ValueError("positions must be [axes][T] with an axis for each the frequencies name")
    if query_out is None:
        query_out = _empty(stream, (T, H, D), dt, query.device, returned=True)
    elif query_out is not query and (query_out.shape != (T, H, D) or query_out.dtype != dt):
        raise ValueError("query_out must match the query")
    st = load_library().pa_rotary_cache_write(
        *_rows(query_out, "query_out", H * D), *_rows(query, "query", H * D),
        *_rows(key, "key", hkv * D), *_rows(value, "value", hkv * D),
        _dev(positions, "positions"), rotary._ptr,
        _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"), _dev(slot_mapping, "slot_mapping"),
        T, nb, bs, H, hkv, d, _dtype_code(dt), _opt_ptr(error_word, "error_word"),
        _stream_ptr(stream, query))
    _check(st, "pa_rotary_cache_write")
    return query_out


def decode_workspace_size(num_seqs: int, num_heads: int, num_kv_heads: int, head_dim: int,
                          max_context_len: int) -> int:
    return int(load_library().pa_decode_workspace_size(num_seqs, num_heads, num_kv_heads,
                                                       head_dim, max_context_len))


def decode_kernel_launches(num_seqs: int, num_heads: int, num_kv_heads: int, head_dim: int,
                           max_context_len: int) -> int:
    """Kernels one decode_attention call enqueues for these sizes."""
    return int(load_library().pa_decode_kernel_launches(num_seqs, num_heads, num_kv_heads,
                                                        head_dim, max_context_len))


def decode_partition_tokens(num_seqs: int, num_kv_heads: int, max_context_len: int) -> int:
    """Partition size pa_decode_attention uses; a merge kernel runs when
    max_context_len exceeds it."""
    return int(load_library().pa_decode_partition_tokens(num_seqs, num_kv_heads,
                                                         max_context_len))


def decode_attention(query, k_cache, v_cache, block_tables, context_lens,
                     max_context_len: int, scale: float, out=None, out_dtype=None,
                     workspace=None, error_word=None, stream=None):
    """Paged decode attention; returns ``out`` [S][H][D] (fp32 unless
    ``out_dtype`` / ``out`` says the input dtype).  ``workspace`` (uint8, >=
    decode_workspace_size bytes) is allocated here when not given.  Pools
    are [num_blocks][Hkv][block_size][D]."""
    torch = _torch()
    S, H, D = query.shape
    nb, hkv, bs, d2 = k_cache.shape
    if d2 != D or v_cache.shape != k_cache.shape:
        raise ValueError("pool shape mismatch")
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise TypeError("block_tables and context_lens must be int32")
    if block_tables.dim() != 2 or block_tables.shape[0] != S or context_lens.shape != (S,):
        raise ValueError("block_tables must be [S][max_blocks], context_lens [S]")
    if out is None:
        out = _empty(stream, (S, H, D), out_dtype or torch.float32, query.device, returned=True)
    if workspace is None:
        nbytes = decode_workspace_size(S, H, hkv, D, int(max_context_len))
        workspace = _workspace(stream, nbytes, query.device)
    head = (_dev(out, "out"), _dtype_code(out.dtype), _dev(query, "query"),
            _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"),
            _dev(block_tables, "block_tables"), block_tables.shape[1],
            _dev(context_lens, "context_lens"), int(max_context_len), S, H, hkv, D, nb)
    tail = (float(scale), _dtype_code(query.dtype), _dev(workspace, "workspace"),
            workspace.numel() * workspace.element_size(), _opt_ptr(error_word, "error_word"),
            _stream_ptr(stream, query))
    lib = load_library()
    if bs == BLOCK_SIZE:
        _check(lib.pa_decode_attention(*head, *tail), "pa_decode_attention")
    else:
        _check(lib.pa_decode_attention_ex(*head, bs, *tail), "pa_decode_attention_ex")
    return out


def decode_attention_contiguous(query, k_cache, v_cache, context_lens, max_context_len: int,
                                scale: float, out=None, out_dtype=None, workspace=None,
                                error_word=None, stream=None):
    """Decode attention over a contiguous (unpaged) cache
    k_cache / v_cache [S][Hkv][max_rows][D] (max_rows a multiple of 16); the
    baseline that measures what the block table costs."""
    torch = _torch()
    S, H, D = query.shape
    s2, hkv, rows, d2 = k_cache.shape
    if s2 != S or d2 != D or v_cache.shape != k_cache.shape:
        raise ValueError("cache shape mismatch")
    if context_lens.dtype != torch.int32 or context_lens.shape != (S,):
        raise TypeError("context_lens must be int32 [S]")
    if out is None:
        out = _empty(stream, (S, H, D), out_dtype or torch.float32, query.device, returned=True)
    if workspace is None:
        nbytes = decode_workspace_size(S, H, hkv, D, int(max_context_len))
        workspace = _workspace(stream, nbytes, query.device)
    st = load_library().pa_decode_attention_contiguous(
        _dev(out, "out"), _dtype_code(out.dtype), _dev(query, "query"), _dev(k_cache, "k_cache"),
        _dev(v_cache, "v_cache"), rows, _dev(context_lens, "context_lens"), int(max_context_len),
        S, H, hkv, D, float(scale), _dtype_code(query.dtype), _dev(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _opt_ptr(error_word, "error_word"),
        _stream_ptr(stream, query))
    _check(st, "pa_decode_attention_contiguous")
    return out


def decode_scored_workspace_size(num_seqs: int, num_heads: int, num_kv_heads: int,
                                 head_dim: int, max_context_len: int) -> int:
    return int(load_library().pa_decode_scored_workspace_size(num_seqs, num_heads, num_kv_heads,
                                                              head_dim, max_context_len))


def _score_rows(scores, rows, name="scores"):
    """Pointer and row stride of fp32 scores [..rows..][stride]."""
    torch = _torch()
    if scores.dtype != torch.float32:
        raise TypeError(f"{name} must be float32")
    shape = scores.shape
    if len(shape) != 3 or shape[:2] != rows:
        raise ValueError(f"{name} must be [S][Hkv][positions]")
    return _dev(scores, name), shape[2]


def decode_attention_scored(query, k_cache, v_cache, block_tables, context_lens,
                            max_context_len: int, scale: float, scores, out=None,
                            out_dtype=None, workspace=None, error_word=None, stream=None):
    """decode_attention that also adds the attention weight each cached token
    received, summed over the query heads of its KV head, to ``scores`` (fp32
    [S][Hkv][>= max_context_len], row s for the batch's sequence s).
    ``workspace`` (uint8, >= decode_scored_workspace_size bytes) is allocated
    here when not given.  Returns ``out``."""
    torch = _torch()
    S, H, D = query.shape
    pool, dt = k_cache.shape, query.dtype
    nb, hkv, bs, d2 = pool
    if d2 != D or v_cache.shape != pool:
        raise ValueError("pool shape mismatch")
    if k_cache.dtype != dt or v_cache.dtype != dt:
        raise ValueError("pools must match the query dtype")
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise TypeError("block_tables and context_lens must be int32")
    tables = block_tables.shape
    if len(tables) != 2 or tables[0] != S or context_lens.shape != (S,):
        raise ValueError("block_tables must be [S][max_blocks], context_lens [S]")
    sc, stride = _score_rows(scores, (S, hkv))
    if out is None:
        out = _empty(stream, (S, H, D), out_dtype or torch.float32, query.device, returned=True)
    elif out.shape != (S, H, D):
        raise ValueError("out must match the query")
    if workspace is None:
        nbytes = decode_scored_workspace_size(S, H, hkv, D, int(max_context_len))
        workspace = _workspace(stream, nbytes, query.device)
    st = load_library().pa_decode_attention_scored(
        _dev(out, "out"), _dtype_code(out.dtype), _dev(query, "query"), _dev(k_cache, "k_cache"),
        _dev(v_cache, "v_cache"), _dev(block_tables, "block_tables"), tables[1],
        _dev(context_lens, "context_lens"), int(max_context_len), S, H, hkv, D, nb, bs,
        float(scale), _dtype_code(dt), sc, stride, _dev(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _opt_ptr(error_word, "error_word"),
        _stream_ptr(stream, query))
    _check(st, "pa_decode_attention_scored")
    return out


def copy_blocks(k_caches: Sequence, v_caches: Sequence, block_pairs, error_word=None,
                stream=None) -> None:
    """For every layer: pools[dst] = pools[src] for each (src, dst) row of
    block_pairs (int64 [P][2], on the device)."""
    torch = _torch()
    if len(k_caches) != len(v_caches) or not k_caches:
        raise ValueError("need the same, non-zero number of K and V pools")
    if block_pairs.dtype != torch.int64:
        raise TypeError("block_pairs must be int64")
    nb, hkv, bs, d = k_caches[0].shape
    for c in list(k_caches) + list(v_caches):
        if c.shape != k_caches[0].shape or c.dtype != k_caches[0].dtype:
            raise ValueError("all pools must have one shape and dtype")
    L = len(k_caches)
    kp = (ctypes.c_void_p * L)(*[_dev(c, "k_caches") for c in k_caches])
    vp = (ctypes.c_void_p * L)(*[_dev(c, "v_caches") for c in v_caches])
    npairs = block_pairs.shape[0] if block_pairs.numel() else 0
    head = (ctypes.cast(kp, ctypes.c_void_p), ctypes.cast(vp, ctypes.c_void_p), L,
            _dev(block_pairs, "block_pairs") if npairs else None, npairs, nb)
    tail = (hkv, d, _dtype_code(k_caches[0].dtype), _opt_ptr(error_word, "error_word"),
            _stream_ptr(stream, k_caches[0]))
    lib = load_library()
    if bs == BLOCK_SIZE:
        _check(lib.pa_copy_blocks(*head, *tail), "pa_copy_blocks")
    else:
        _check(lib.pa_copy_blocks_ex(*head, bs, *tail), "pa_copy_blocks_ex")


def _pool_ptr(t, name):
    """Pool pointer for pa_swap_blocks: a CUDA tensor or a pinned CPU tensor."""
    if not (t.is_cuda or t.is_pinned()):
        raise ValueError(f"{name} must be a CUDA tensor or pinned host memory")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def swap_blocks(dst_k_caches: Sequence, dst_v_caches: Sequence, src_k_caches: Sequence,
                src_v_caches: Sequence, block_pairs, error_word=None, stream=None) -> None:
    """For every layer: dst[pair dst] = src[pair src] for each (src, dst) row
    of block_pairs (int64 [P][2], on the device).  Pools are
    [num_blocks][Hkv][block_size][D]; either side may be device memory or
    pinned host memory (the CPU swap space)."""
    torch = _torch()
    L = len(dst_k_caches)
    if not (L == len(dst_v_caches) == len(src_k_caches) == len(src_v_caches)) or not L:
        raise ValueError("need the same, non-zero number of pools on each side")
    if block_pairs.dtype != torch.int64:
        raise TypeError("block_pairs must be int64")
    nd, hkv, bs, d = dst_k_caches[0].shape
    ns = src_k_caches[0].shape[0]
    dt = dst_k_caches[0].dtype
    for c in list(dst_k_caches) + list(dst_v_caches):
        if tuple(c.shape) != (nd, hkv, bs, d) or c.dtype != dt:
            raise ValueError("destination pools must have one shape and dtype")
    for c in list(src_k_caches) + list(src_v_caches):
        if tuple(c.shape) != (ns, hkv, bs, d) or c.dtype != dt:
            raise ValueError("source pools must match the destination's block shape and dtype")
    arr = lambda xs, n: ctypes.cast((ctypes.c_void_p * L)(*[_pool_ptr(x, n) for x in xs]),
                                    ctypes.c_void_p)
    npairs = block_pairs.shape[0] if block_pairs.numel() else 0
    on_gpu = next((c for c in [block_pairs] + list(dst_k_caches) + list(src_k_caches)
                   if c.is_cuda), None)
    st = load_library().pa_swap_blocks(
        arr(dst_k_caches, "dst_k_caches"), arr(dst_v_caches, "dst_v_caches"),
        arr(src_k_caches, "src_k_caches"), arr(src_v_caches, "src_v_caches"), L,
        block_pairs.data_ptr() if npairs else None, npairs, nd, ns, bs, hkv, d, _dtype_code(dt),
        _opt_ptr(error_word, "error_word"), _stream_ptr(stream, on_gpu))
    _check(st, "pa_swap_blocks")


def prefill_workspace_size(num_seqs: int, num_heads: int, num_kv_heads: int, head_dim: int,
                           max_query_len: int) -> int:
    return int(load_library().pa_prefill_workspace_size(num_seqs, num_heads, num_kv_heads,
                                                        head_dim, max_query_len))


def prefill_attention(query, k_cache, v_cache, block_tables, query_start_loc, context_lens,
                      max_query_len: int, max_context_len: int, scale: float, out=None,
                      out_dtype=None, workspace=None, error_word=None, stream=None, lse=None):
    """Chunked-prefill attention: query [T][H][D] holds every sequence's new
    tokens (sequence s: rows query_start_loc[s] .. query_start_loc[s+1]-1),
    already written to the cache as its last positions; context_lens[s]
    counts the tokens after the chunk.  ``workspace`` (uint8, >=
    prefill_workspace_size bytes) is allocated here when not given.  ``lse``
    (fp32 [T][H], optional) gets each row's log-sum-exp.  Returns out
    [T][H][D]."""
    torch = _torch()
    T, H, D = query.shape
    nb, hkv, bs, d2 = k_cache.shape
    if d2 != D or v_cache.shape != k_cache.shape:
        raise ValueError("pool shape mismatch")
    for t, n in ((block_tables, "block_tables"), (query_start_loc, "query_start_loc"),
                 (context_lens, "context_lens")):
        if t.dtype != torch.int32:
            raise TypeError(f"{n} must be int32")
    S = context_lens.shape[0]
    if query_start_loc.shape != (S + 1,) or block_tables.dim() != 2 or \
            block_tables.shape[0] != S:
        raise ValueError("query_start_loc must be [S+1], block_tables [S][max_blocks]")
    if out is None:
        out = _empty(stream, (T, H, D), out_dtype or torch.float32, query.device, returned=True)
    if workspace is None:
        nbytes = prefill_workspace_size(S, H, hkv, D, int(max_query_len))
        workspace = _workspace(stream, nbytes, query.device)
    head = (_dev(out, "out"), _dtype_code(out.dtype), _dev(query, "query"),
            _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"),
            _dev(block_tables, "block_tables"), block_tables.shape[1],
            _dev(query_start_loc, "query_start_loc"), _dev(context_lens, "context_lens"),
            int(max_query_len), int(max_context_len), S, T, H, hkv, D, nb, bs, float(scale),
            _dtype_code(query.dtype))
    tail = (_dev(workspace, "workspace"), workspace.numel() * workspace.element_size(),
            _opt_ptr(error_word, "error_word"), _stream_ptr(stream, query))
    lib = load_library()
    if lse is None:
        _check(lib.pa_prefill_attention(*head, *tail), "pa_prefill_attention")
    else:
        _check(lib.pa_prefill_attention_lse(*head, _lse_ptr(lse, T, H), *tail),
               "pa_prefill_attention_lse")
    return out


def _lse_ptr(lse, T, H):
    torch = _torch()
    if lse.dtype != torch.float32 or tuple(lse.shape) != (T, H):
        raise ValueError("lse must be float32 [T][H]")
    return _dev(lse, "lse")


def prefill_scores_workspace_size(num_seqs: int, num_heads: int, num_kv_heads: int,
                                  head_dim: int, max_query_len: int,
                                  max_context_len: int) -> int:
    return int(load_library().pa_prefill_scores_workspace_size(
        num_seqs, num_heads, num_kv_heads, head_dim, max_query_len, max_context_len))


def prefill_scores(query, lse, k_cache, block_tables, query_start_loc, context_lens,
                   max_query_len: int, max_context_len: int, scale: float, scores,
                   workspace=None, error_word=None, stream=None):
    """Add the attention weight that each sequence's query rows (rows
    query_start_loc[s] .. query_start_loc[s+1]-1 of query [T][H][D], its last
    positions: a prompt, a chunk or a window) give to its cached tokens to
    ``scores`` (fp32 [S][Hkv][>= max_context_len]).  ``lse`` [T][H] is the rows'
    log-sum-exp (prefill_attention's).  No ``workspace`` is needed (one of
    prefill_scores_workspace_size bytes is accepted).  Returns ``scores``."""
    torch = _torch()
    T, H, D = query.shape
    nb, hkv, bs, d2 = k_cache.shape
    if d2 != D or k_cache.dtype != query.dtype:
        raise ValueError("the pool must match the query")
    for t, n in ((block_tables, "block_tables"), (query_start_loc, "query_start_loc"),
                 (context_lens, "context_lens")):
        if t.dtype != torch.int32:
            raise TypeError(f"{n} must be int32")
    S = context_lens.shape[0]
    if query_start_loc.shape != (S + 1,) or block_tables.dim() != 2 or \
            block_tables.shape[0] != S:
        raise ValueError("query_start_loc must be [S+1], block_tables [S][max_blocks]")
    sc, stride = _score_rows(scores, (S, hkv))
    ws = (None, 0) if workspace is None else (
        _dev(workspace, "workspace"), workspace.numel() * workspace.element_size())
    st = load_library().pa_prefill_scores(
        _dev(query, "query"), _lse_ptr(lse, T, H), _dev(k_cache, "k_cache"),
        _dev(block_tables, "block_tables"), block_tables.shape[1],
        _dev(query_start_loc, "query_start_loc"), _dev(context_lens, "context_lens"),
        int(max_query_len), int(max_context_len), S, T, H, hkv, D, nb, bs, float(scale),
        _dtype_code(query.dtype), sc, stride, *ws, _opt_ptr(error_word, "error_word"),
        _stream_ptr(stream, query))
    _check(st, "pa_prefill_scores")
    return scores


def evict_workspace_size(num_layers: int, num_seqs: int, num_kv_heads: int, max_context_len: int,
                         max_keep_len: int) -> int:
    return int(load_library().pa_evict_workspace_size(num_layers, num_seqs, num_kv_heads,
                                                      max_context_len, max_keep_len))


def _layer_ptrs(xs, name, num_layers, shape, dtype):
    """Pointers of one tensor a layer, all of one shape and dtype."""
    if len(xs) != num_layers:
        raise ValueError(f"need one {name} per layer")
    ptrs = []
    for x in xs:
        if x.shape != shape or x.dtype != dtype:
            raise ValueError(f"{name} must be {dtype} {list(shape)} in every layer")
        ptrs.append(_dev(x, name))
    return ptrs


def evict_tokens(k_caches: Sequence, v_caches: Sequence, scores: Sequence, block_tables,
                 context_lens, keep_lens, max_context_len: int, max_keep_len: int,
                 num_sink: int = 0, num_recent: int = 0, dst_block_tables=None,
                 scores_out: Optional[Sequence] = None, kept: Optional[Sequence] = None,
                 new_lens=None, workspace=None, error_word=None, stream=None):
    """Shrink every sequence s to min(context_lens[s], keep_lens[s]) tokens in
    every layer: each KV head keeps the first num_sink, the last num_recent
    and the highest-scored tokens between them, in their order (equal scores:
    the lowest index), and K, V and the scores are compacted onto them.

    k_caches, v_caches, scores: one per layer; scores fp32 [S][Hkv][>=
    max_context_len], vacated positions become zero.  In place unless
    dst_block_tables (int32 [S][blocks], blocks no source table names) says
    where K and V go and scores_out (one per layer) where the scores go.
    kept (int32 [S][Hkv][>= max_keep_len] per layer) gets the kept tokens'
    positions.  max_keep_len bounds the lengths left.  ``workspace`` (uint8,
    >= evict_workspace_size bytes) is allocated here when not given.  Returns
    new_lens, int32 [S]."""
    torch = _torch()
    L = len(k_caches)
    if not L or len(v_caches) != L or len(scores) != L:
        raise ValueError("need the same, non-zero number of K pools, V pools and scores")
    pool, dt = k_caches[0].shape, k_caches[0].dtype
    nb, hkv, bs, d = pool
    i32 = torch.int32
    if block_tables.dtype != i32 or context_lens.dtype != i32 or keep_lens.dtype != i32:
        raise TypeError("block_tables, context_lens and keep_lens must be int32")
    S = context_lens.shape[0]
    tables = block_tables.shape
    if len(tables) != 2 or tables[0] != S or context_lens.shape != (S,) or \
            keep_lens.shape != (S,):
        raise ValueError("block_tables must be [S][max_blocks], context_lens and keep_lens [S]")
    dst = (S, 0) if dst_block_tables is None else dst_block_tables.shape
    if len(dst) != 2 or dst[0] != S or (
            dst_block_tables is not None and dst_block_tables.dtype != i32):
        raise ValueError("dst_block_tables must be int32 [S][blocks]")

    # the layers' pointers, one array after the other
    ptrs = _layer_ptrs(k_caches, "k_caches", L, pool, dt)
    ptrs += _layer_ptrs(v_caches, "v_caches", L, pool, dt)

    def rows(xs, name, dtype):  # [S][Hkv][positions]: where its array is, positions
        first = xs[0].shape if len(xs) else ()
        if len(first) != 3 or first[0] != S or first[1] != hkv:
            raise ValueError(f"{name} must be {dtype} [S][Hkv][positions] in every layer")
        ptrs.extend(_layer_ptrs(xs, name, L, first, dtype))
        return len(ptrs) - L, first[2]

    sc = rows(scores, "scores", torch.float32)
    out = None if scores_out is None else rows(scores_out, "scores_out", torch.float32)
    kp = None if kept is None else rows(kept, "kept", i32)
    arrays = array.array("Q", ptrs)
    base = arrays.buffer_info()[0]
    none = (None, 0)
    if new_lens is None:
        new_lens = _empty(stream, S, torch.int32, context_lens.device, returned=True)
    elif new_lens.dtype != torch.int32 or new_lens.shape != (S,):
        raise ValueError("new_lens must be int32 [S]")
    if workspace is None:
        nbytes = evict_workspace_size(L, S, hkv, int(max_context_len), int(max_keep_len))
        workspace = _workspace(stream, nbytes, context_lens.device)
    st = load_library().pa_evict_tokens(
        base, base + 8 * L, L, base + 8 * sc[0], sc[1],
        *(none if out is None else (base + 8 * out[0], out[1])),
        *(none if kp is None else (base + 8 * kp[0], kp[1])),
        _dev(block_tables, "block_tables"), tables[1],
        _opt_ptr(dst_block_tables, "dst_block_tables"), dst[1],
        _dev(context_lens, "context_lens"), _dev(keep_lens, "keep_lens"),
        _dev(new_lens, "new_lens"), int(max_context_len), int(max_keep_len), int(num_sink),
        int(num_recent), S, nb, bs, hkv, d, _dtype_code(dt), _dev(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _opt_ptr(error_word, "error_word"),
        _stream_ptr(stream, k_caches[0]))
    _check(st, "pa_evict_tokens")
    return new_lens
