"""ctypes binding of include/prefill_attn.h (argument marshalling only).

Every function here has the name of the C entry point it calls.  Tensors are
PyTorch CUDA tensors; their data pointers, sizes and the current CUDA stream
are passed straight to the library, which does all of the work on the GPU.
There is no fallback: if the compiled library is missing, loading fails.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

from . import build as _build

PA_OK = 0
STATUS = {0: "PA_OK", 1: "PA_ERR_INVALID_ARG", 2: "PA_ERR_UNSUPPORTED", 3: "PA_ERR_CUDA",
          4: "PA_ERR_DEVICE_TIMEOUT", 5: "PA_ERR_DEVICE_METADATA", 6: "PA_ERR_DEVICE_LAYOUT"}
DEVERR_METADATA, DEVERR_TIMEOUT, DEVERR_OVERFLOW, DEVERR_SMEM_ALIGN = 0x1, 0x2, 0x4, 0x8

class PaOptions(ctypes.Structure):
    """pa_options of include/prefill_attn.h."""
    _fields_ = [("struct_size", ctypes.c_uint32), ("window", ctypes.c_int32),
                ("block_table", ctypes.c_void_p), ("block_size", ctypes.c_int32),
                ("max_blocks_per_seq", ctypes.c_int32), ("num_blocks", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("rope_theta", ctypes.c_float), ("reserved2", ctypes.c_int32),
                ("kv_quant", ctypes.c_int32), ("reserved3", ctypes.c_int32),
                ("cache_k_scale", ctypes.c_void_p), ("cache_v_scale", ctypes.c_void_p),
                ("wait_timeout_test", ctypes.c_int32), ("schedule", ctypes.c_int32)]


class PaPrefix(ctypes.Structure):
    """pa_prefix of include/prefill_attn.h."""
    _fields_ = [("struct_size", ctypes.c_uint32), ("len", ctypes.c_int32), ("k", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("capacity", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("block_table", ctypes.c_void_p)]


class PaCache4(ctypes.Structure):
    """pa_cache4 of include/prefill_attn.h."""
    _fields_ = [("struct_size", ctypes.c_uint32), ("group", ctypes.c_int32), ("k", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("k_params", ctypes.c_void_p), ("v_params", ctypes.c_void_p)]


# Entry points declared in include/prefill_attn.h: name -> (restype, argtypes)
_P, _I, _F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
_VARLEN_ARGS = [_P] * 10 + [_I] * 6 + [_F, _I, _P]
_VARLEN_EX_ARGS = [_P] * 10 + [_I] * 6 + [_F, _I, ctypes.POINTER(PaOptions), _P]
SIGNATURES = {
    "prefill_attn_varlen": (_I, _VARLEN_ARGS),
    "prefill_attn_varlen_validate": (_I, _VARLEN_ARGS),
    "prefill_attn_varlen_noalloc": (_I, _VARLEN_ARGS),
    "prefill_attn_varlen_ex": (_I, _VARLEN_EX_ARGS),
    "prefill_attn_varlen_sinks": (_I, [_P] * 10 + [_I] * 6 + [_F, _I, ctypes.POINTER(PaOptions), _P]),
    "prefill_attn_varlen_prefix": (_I, [_P] * 10 + [_I] * 6 + [_F, _I, ctypes.POINTER(PaPrefix),
                                                              ctypes.POINTER(PaOptions), _P]),
    "prefill_attn_key_weights": (_I, [_P] * 8 + [_I] * 6 + [_F, _I, _I, _I, ctypes.POINTER(PaOptions), _P]),
    "prefill_attn_evict": (_I, [_P] * 7 + [_I] * 7 + [ctypes.POINTER(PaOptions), _P]),
    "prefill_attn_varlen_cache4": (_I, [_P] * 5 + [ctypes.POINTER(PaCache4)] + [_P] * 3 + [_I] * 6
                                   + [_F, _I, ctypes.POINTER(PaOptions), _P]),
    "prefill_attn_cache4_write": (_I, [_P] * 3 + [ctypes.POINTER(PaCache4), _P] + [_I] * 5
                                  + [ctypes.POINTER(PaOptions), _P]),
    "prefill_attn_cache4_read": (_I, [ctypes.POINTER(PaCache4)] + [_P] * 4 + [_I] * 5 + [ctypes.POINTER(PaOptions), _P]),
    "prefill_attn_device_status": (_I, [_P, ctypes.POINTER(ctypes.c_int32)]),
    "prefill_attn_release": (None, []),
    "prefill_attn_status_string": (ctypes.c_char_p, [_I]),
    "prefill_attn_last_error": (ctypes.c_char_p, []),
    "prefill_attn_last_launch_count": (_I, []),
    "prefill_attn_last_schedule": (_I, []),
    "prefill_attn_auto_schedule": (_I, [_I, _I, _I, _I, _I, _I]),
}

_lib = None


class PrefillAttnError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


def library_path() -> str:
    return _build.LIB_PATH


def load(path: Optional[str] = None):
    """Load (once) the compiled library and bind every declared entry point."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or library_path()
    if not os.path.exists(p):
        raise RuntimeError(f"prefill_attn library not built: {p} is missing "
                           "(run prefill_phase_attention_gb300.build.build())")
    lib = ctypes.CDLL(p)
    for name, (res, args) in SIGNATURES.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    if path is None:
        _lib = lib
    return lib


def _check(status: int):
    if status != PA_OK:
        raise PrefillAttnError(status, load().prefill_attn_last_error().decode())


# The current stream's raw handle: torch's own accessor costs ~0.1 us, building
# a torch.cuda.Stream object for it ~3 us (a quarter of a small call's host time).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_handle(stream, device_index: Optional[int] = None) -> int:
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None and device_index is not None:
        return _raw_stream(device_index)
    return torch.cuda.current_stream().cuda_stream


def _varlen_args(q, k, v, cu_seqlens_q, cu_seqlens_k, cache_k, cache_v, cache_offsets, out, lse,
                 scale, causal, stream, max_cache_len=None, cache_dtype=torch.bfloat16):
    for name, t, dt in (("q", q, torch.bfloat16), ("k", k, torch.bfloat16), ("v", v, torch.bfloat16),
                        ("cache_k", cache_k, cache_dtype), ("cache_v", cache_v, cache_dtype),
                        ("out", out, torch.bfloat16), ("cu_seqlens_q", cu_seqlens_q, torch.int32),
                        ("cu_seqlens_k", cu_seqlens_k, torch.int32), ("cache_offsets", cache_offsets, torch.int32)):
        if t.dtype != dt or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA {dt} tensor")
    if lse is not None and (lse.dtype != torch.float32 or not lse.is_cuda or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous CUDA float32 tensor")
    if q.dim() != 3 or k.dim() != 3 or cache_k.dim() != 4:
        raise ValueError("q/k/v are [total_q, heads, head_dim]; caches are [num_seqs, kv_heads, cap, head_dim]")
    total_q, n_heads, head_dim = q.shape
    n_kv_heads = k.shape[1]
    num_seqs = cache_offsets.numel()
    if scale is None:
        scale = head_dim ** -0.5
    return (q.data_ptr(), k.data_ptr(), v.data_ptr(), cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(),
            cache_k.data_ptr(), cache_v.data_ptr(), cache_offsets.data_ptr(), out.data_ptr(),
            None if lse is None else lse.data_ptr(),
            num_seqs, total_q, cache_k.shape[2] if max_cache_len is None else max_cache_len,
            n_heads, n_kv_heads, head_dim,
            float(scale), int(bool(causal)), _stream_handle(stream, q.get_device()))


def prefill_attn_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, cache_k, cache_v, cache_offsets, out,
                        lse=None, *, scale: Optional[float] = None, causal: bool = True, stream=None) -> None:
    """Enqueue causal varlen prefill attention + the KV-cache write on `stream`.

    Shapes: q/out [total_q, n_heads, head_dim], k/v [total_q, n_kv_heads, head_dim] (bf16),
    cache_k/v [num_seqs, n_kv_heads, max_cache_len, head_dim] (bf16), cu_seqlens_q/k
    [num_seqs+1], cache_offsets [num_seqs] (int32), lse [total_q, n_heads] fp32 or None.
    """
    args = _varlen_args(q, k, v, cu_seqlens_q, cu_seqlens_k, cache_k, cache_v, cache_offsets, out, lse,
                        scale, causal, stream)
    _check(load().prefill_attn_varlen(*args))


def make_options(window: int = 0, block_table=None, block_size: int = 0, num_blocks: int = 0,
                 rope_theta: float = 0.0, cache_k_scale=None, cache_v_scale=None,
                 wait_timeout_test: bool = False, schedule: int = 0) -> PaOptions:
    o = PaOptions()
    o.struct_size = ctypes.sizeof(PaOptions)
    o.window = int(window)
    o.rope_theta = float(rope_theta)
    o.wait_timeout_test = int(bool(wait_timeout_test))
    o.schedule = int(schedule)
    if cache_k_scale is not None:
        o.kv_quant = 1
        o.cache_k_scale = cache_k_scale.data_ptr()
        o.cache_v_scale = cache_v_scale.data_ptr()
    if block_table is not None:
        o.block_table = block_table.data_ptr()
        o.block_size = int(block_size)
        o.max_blocks_per_seq = int(block_table.shape[1])
        o.num_blocks = int(num_blocks)
    return o


def _cache_args(cache_k, block_table, cache_k_scale, cache_v_scale):
    """Checks the cache options; returns (slot capacity of a paged cache or None, whether the cache is int8)."""
    cap = None
    if block_table is not None:
        if block_table.dtype != torch.int32 or not block_table.is_cuda or not block_table.is_contiguous() \
                or block_table.dim() != 2:
            raise ValueError("block_table must be a contiguous 2-D CUDA int32 tensor")
        cap = block_table.shape[1] * cache_k.shape[2]
    quant = cache_k_scale is not None or cache_v_scale is not None
    if quant:
        for name, t in (("cache_k_scale", cache_k_scale), ("cache_v_scale", cache_v_scale)):
            if t is None or t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous() \
                    or tuple(t.shape) != tuple(cache_k.shape[:-1]):
                raise ValueError(f"{name} must be a contiguous CUDA float32 tensor of shape cache.shape[:-1]")
    return cap, quant


def prefill_attn_varlen_ex(q, k, v, cu_seqlens_q, cu_seqlens_k, cache_k, cache_v, cache_offsets, out, lse=None, *,
                           scale: Optional[float] = None, causal: bool = True, window: int = 0,
                           block_table=None, rope_theta: float = 0.0, cache_k_scale=None, cache_v_scale=None,
                           wait_timeout_test: bool = False, schedule: int = 0, stream=None) -> None:
    """prefill_attn_varlen with options.

    window > 0 restricts each query to its `window` most recent keys (causal only).
    block_table (int32 CUDA [num_seqs, max_blocks_per_seq]) selects the paged cache:
    cache_k/v are then block pools [num_blocks, n_kv_heads, block_size, head_dim]
    and position p of sequence b lives in row p % block_size of block
    block_table[b, p // block_size].
    rope_theta > 0 rotates every new q/k to its absolute position (rotary
    embedding, rotate-half pairing) before attention and the cache write.
    cache_k_scale / cache_v_scale (fp32 CUDA [num_seqs, n_kv_heads, max_cache_len])
    select the int8 cache: cache_k/v are then int8 codes and row (b, h, p) stands
    for code * scale.
    schedule fixes the work schedule (pa_options.schedule: 1 one-tile units
    splitting their KV tiles between the two slots, 2 two-tile units, 3
    two-tile units with single-tile ones split; 0 = the library's choice).
    """
    cap, quant = _cache_args(cache_k, block_table, cache_k_scale, cache_v_scale)
    args = _varlen_args(q, k, v, cu_seqlens_q, cu_seqlens_k, cache_k, cache_v, cache_offsets, out, lse,
                        scale, causal, stream, max_cache_len=cap,
                        cache_dtype=torch.int8 if quant else torch.bfloat16)
    opts = make_options(window, block_table, cache_k.shape[2], cache_k.shape[0], rope_theta,
                        cache_k_scale, cache_v_scale, wait_timeout_test, schedule)
    _check(load().prefill_attn_varlen_ex(*args[:-1], ctypes.byref(opts), args[-1]))


# The long-context calls are often a few microseconds of GPU work, so their checks
# read as few attributes as they need, as one expression where every call goes
# through (0.3 us a tensor on the GPU's host; _check_tensors then names the
# tensor that failed).  Tensors have the shapes that their documentation states;
# of the vectors of metadata the element count says whether they fit.
_BF16, _I8, _F32, _I32 = torch.bfloat16, torch.int8, torch.float32, torch.int32
_INT = 0x7fffffff


def _check_tensors(device: int, *specs) -> None:
    """Each spec (name, tensor or None, dtype, shape, or the elements of a vector): contiguous, CUDA, on `device`, of
    that type and shape."""
    for name, t, dtype, n in specs:
        if t is not None and (t.dtype is not dtype or t.get_device() != device or not t.is_contiguous()
                              or (t.numel() != n if type(n) is int else t.shape != n)):
            size = f"of {n} elements" if type(n) is int else f"of shape {tuple(n)}"
            raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor {size} on cuda:{device}, "
                             f"not {t.dtype} {tuple(t.shape)} on {t.device}")


def _current_device(q) -> int:
    """The index of q's device, which must be the current one (the library launches there)."""
    device = q.get_device()
    if device < 0:
        raise ValueError("tensors must be CUDA tensors")
    if device != torch._C._cuda_getDevice():
        raise ValueError(f"tensors on cuda:{device}, but the current device is cuda:{torch._C._cuda_getDevice()}")
    return device


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream_on(stream, device: int) -> int:
    if stream is None:
        return _raw_stream(device) if _raw_stream is not None else _stream_handle(None, device)
    if stream.device_index != device:
        raise ValueError(f"the stream is on cuda:{stream.device_index}, the tensors on cuda:{device}")
    return stream.cuda_stream


def _cache_specs(device, cache_k, cache_v, b, block_table, cache_k_scale, cache_v_scale, hk, d):
    """Checks a call's cache tensors; returns (slot capacity, whether the cache is int8, shape of the cache's rows)."""
    if cache_k.dim() != 4:
        raise ValueError("caches are [num_seqs, kv_heads, cap, head_dim], or [num_blocks, kv_heads, block_size, head_dim]")
    shape = cache_k.shape
    n, ck_heads, rows, ck_dim = shape
    if ck_heads != hk or ck_dim != d or (block_table is None and n != b):
        raise ValueError(f"cache_k has shape {tuple(cache_k.shape)}: {hk} KV heads of {d}"
                         + ("" if block_table is not None else f" in {b} slots") + " are wanted")
    dtype, quant, cap, total = _BF16, False, rows, (n, hk, rows)
    if block_table is not None:
        if block_table.dim() != 2 or block_table.shape[0] != b:
            raise ValueError(f"block_table must be [{b}, max_blocks_per_seq]")
        cap = block_table.shape[1] * rows
        _check_tensors(device, ("block_table", block_table, _I32, block_table.numel()))
    if cache_k_scale is not None or cache_v_scale is not None:
        if cache_k_scale is None or cache_v_scale is None:
            raise ValueError("an int8 cache needs both cache_k_scale and cache_v_scale")
        dtype, quant = _I8, True
        _check_tensors(device, ("cache_k_scale", cache_k_scale, _F32, total), ("cache_v_scale", cache_v_scale, _F32, total))
    cv = cache_k if cache_v is None else cache_v
    if not (cache_k.dtype is dtype and cache_k.is_contiguous() and cache_k.get_device() == device
            and cv.dtype is dtype and cv.shape == shape and cv.is_contiguous() and cv.get_device() == device):
        _check_tensors(device, ("cache_k", cache_k, dtype, shape), ("cache_v", cache_v, dtype, shape))
    return cap, quant, total


def _attention_args(q, k, v, cu_seqlens_q, cu_seqlens_k, cache_k, cache_v, cache_offsets, out, lse, block_table,
                    cache_k_scale, cache_v_scale):
    """Checks the tensors of a long-context call; returns (device, cache capacity, whether it is int8, its rows' shape)."""
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q/k/v are [total_q, heads, head_dim]")
    device = _current_device(q)
    q_shape, k_shape, b = q.shape, k.shape, cache_offsets.numel()
    (t, h, d), (kt, hk, kd) = q_shape, k_shape
    if kt != t or kd != d:
        raise ValueError(f"k has shape {tuple(k_shape)}, q {tuple(q_shape)}")
    vv, oo = k if v is None else v, q if out is None else out
    if not (q.dtype is _BF16 and k.dtype is _BF16 and q.is_contiguous() and k.is_contiguous() and k.get_device() == device
            and vv.dtype is _BF16 and vv.shape == k_shape and vv.is_contiguous() and vv.get_device() == device
            and oo.dtype is _BF16 and oo.shape == q_shape and oo.is_contiguous() and oo.get_device() == device
            and (lse is None or lse.dtype is _F32 and lse.shape == (t, h) and lse.is_contiguous()
                 and lse.get_device() == device)
            and cu_seqlens_q.dtype is _I32 and cu_seqlens_q.numel() == b + 1 and cu_seqlens_q.is_contiguous()
            and cu_seqlens_q.get_device() == device
            and cu_seqlens_k.dtype is _I32 and cu_seqlens_k.numel() == b + 1 and cu_seqlens_k.is_contiguous()
            and cu_seqlens_k.get_device() == device
            and cache_offsets.dtype is _I32 and cache_offsets.is_contiguous() and cache_offsets.get_device() == device):
        _check_tensors(device, ("q", q, _BF16, q_shape), ("k", k, _BF16, k_shape), ("v", v, _BF16, k_shape),
                       ("out", out, _BF16, q_shape), ("lse", lse, _F32, (t, h)), ("cu_seqlens_q", cu_seqlens_q, _I32, b + 1),
                       ("cu_seqlens_k", cu_seqlens_k, _I32, b + 1), ("cache_offsets", cache_offsets, _I32, b))
    return device, *_cache_specs(device, cache_k, cache_v, b, block_table, cache_k_scale, cache_v_scale, hk, d)


def _pointers(q, k, v, cu_seqlens_q, cu_seqlens_k, cache_k, cache_v, cache_offsets, out, lse, cap, scale):
    t, h, d = q.shape
    return (q.data_ptr(), k.data_ptr(), v.data_ptr(), cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(),
            cache_k.data_ptr(), cache_v.data_ptr(), cache_offsets.data_ptr(), out.data_ptr(), _ptr(lse),
            cache_offsets.numel(), t, cap, h, k.shape[1], d, d ** -0.5 if scale is None else scale)


def _int32(**values) -> None:
    """The C calls take 32-bit integers, and ctypes cuts larger ones off without a word."""
    for name, v in values.items():
        if v > _INT or v < -_INT - 1:
            raise ValueError(f"{name} = {v} does not fit 32 bits")


def _unread(why: str, **tensors) -> None:
    for name, t in tensors.items():
        if t is not None:
            raise ValueError(f"{why}: {name} would not be read")


def _options(cache_k, block_table, cache_k_scale, cache_v_scale, window=0, rope_theta=0.0, schedule=0):
    """pa_options by position (struct_size, window, block_table, block_size, max_blocks_per_seq, num_blocks, ...)."""
    paged, quant = block_table is not None, cache_k_scale is not None
    return PaOptions(_OPTIONS_SIZE, window, block_table.data_ptr() if paged else None,
                     cache_k.shape[2] if paged else 0, block_table.shape[1] if paged else 0,
                     cache_k.shape[0] if paged else 0, 0, rope_theta, 0, 1 if quant else 0, 0,
                     cache_k_scale.data_ptr() if quant else None, cache_v_scale.data_ptr() if quant else None, 0, schedule)


_OPTIONS_SIZE, _PREFIX_SIZE = ctypes.sizeof(PaOptions), ctypes.sizeof(PaPrefix)


def prefill_attn_varlen_sinks(q, k, v, cu_seqlens_q, cu_seqlens_k, cache_k, cache_v, cache_offsets, out, lse=None, *,
                              window: int, sink_tokens: int, scale: Optional[float] = None, block_table=None,
                              rope_theta: float = 0.0, cache_k_scale=None, cache_v_scale=None, schedule: int = 0,
                              stream=None) -> None:
    """Causal attention under a sliding window whose first `sink_tokens` keys stay visible.

    The query at absolute position p sees key j when j <= p and (j > p - window or
    j < sink_tokens).  Tensors and options as in prefill_attn_varlen_ex.
    """
    if not (-1 <= window <= _INT and -1 <= sink_tokens <= _INT):
        _int32(window=window, sink_tokens=sink_tokens)
    device, cap, _, _ = _attention_args(q, k, v, cu_seqlens_q, cu_seqlens_k, cache_k, cache_v, cache_offsets, out, lse,
                                        block_table, cache_k_scale, cache_v_scale)
    _check((_lib or load()).prefill_attn_varlen_sinks(
        *_pointers(q, k, v, cu_seqlens_q, cu_seqlens_k, cache_k, cache_v, cache_offsets, out, lse, cap, scale),
        sink_tokens, _options(cache_k, block_table, cache_k_scale, cache_v_scale, window, rope_theta, schedule),
        _stream_on(stream, device)))


def prefill_attn_varlen_prefix(q, k, v, cu_seqlens_q, cu_seqlens_k, cache_k, cache_v, cache_offsets, out, lse=None, *,
                               prefix_k=None, prefix_v=None, prefix_len: Optional[int] = None, prefix_table=None,
                               prefix_k_scale=None, prefix_v_scale=None, scale: Optional[float] = None,
                               causal: bool = True, block_table=None, rope_theta: float = 0.0, cache_k_scale=None,
                               cache_v_scale=None, schedule: int = 0, stream=None) -> None:
    """Attention for a batch whose sequences all start with the same prefix, read once.

    Contiguous cache: prefix_k / prefix_v [n_kv_heads, capacity, head_dim] hold the prefix's
    keys and values in their first prefix_len rows (default: all of them), with fp32
    prefix_k_scale / prefix_v_scale [n_kv_heads, capacity] for an int8 cache.  Paged cache:
    prefix_table (int32 CUDA, one entry per block) names the prefix's blocks in the pools,
    and prefix_len its tokens.  A tensor of the other kind is refused.  cu_seqlens_k and
    cache_offsets count each sequence's own tokens, which follow the prefix.
    """
    paged = block_table is not None
    if paged and not (prefix_k is prefix_v is prefix_k_scale is prefix_v_scale is None):
        _unread("a paged cache's prefix is in its pools (prefix_table, prefix_len)", prefix_k=prefix_k, prefix_v=prefix_v,
                prefix_k_scale=prefix_k_scale, prefix_v_scale=prefix_v_scale)
    if not paged and prefix_table is not None:
        _unread("a contiguous cache's prefix is prefix_k and prefix_v", prefix_table=prefix_table)
    if cache_k_scale is None and not (prefix_k_scale is prefix_v_scale is None):
        _unread("a bf16 cache's prefix has no scales", prefix_k_scale=prefix_k_scale, prefix_v_scale=prefix_v_scale)
    device, cap, quant, _ = _attention_args(q, k, v, cu_seqlens_q, cu_seqlens_k, cache_k, cache_v, cache_offsets, out,
                                            lse, block_table, cache_k_scale, cache_v_scale)
    if paged:
        if prefix_table is None or prefix_len is None:
            raise ValueError("a paged cache needs prefix_table and prefix_len")
        _check_tensors(device, ("prefix_table", prefix_table, _I32, prefix_table.numel()))
        if prefix_len > prefix_table.numel() * cache_k.shape[2]:
            raise ValueError("prefix_table has fewer blocks than prefix_len needs")
        _int32(prefix_len=prefix_len)
        pre = PaPrefix(_PREFIX_SIZE, prefix_len, None, None, 0, 0, None, None, prefix_table.data_ptr())
    else:
        if prefix_k is None or prefix_v is None:
            raise ValueError("a contiguous cache needs prefix_k and prefix_v")
        shape, dtype = prefix_k.shape, _I8 if quant else _BF16
        if len(shape) != 3 or shape[0] != k.shape[1] or shape[2] != q.shape[2]:
            raise ValueError("prefix_k is [n_kv_heads, capacity, head_dim]")
        if not (prefix_k.dtype is dtype and prefix_k.is_contiguous() and prefix_k.get_device() == device
                and prefix_v.dtype is dtype and prefix_v.shape == shape and prefix_v.is_contiguous()
                and prefix_v.get_device() == device):
            _check_tensors(device, ("prefix_k", prefix_k, dtype, shape), ("prefix_v", prefix_v, dtype, shape))
        if quant:
            for name, t in (("prefix_k_scale", prefix_k_scale), ("prefix_v_scale", prefix_v_scale)):
                if t is None:
                    raise ValueError(f"an int8 cache needs {name}")
                _check_tensors(device, (name, t, _F32, shape[:2]))
        if prefix_len is None:
            prefix_len = shape[1]
        if not -1 <= prefix_len <= _INT:
            _int32(prefix_len=prefix_len)
        pre = PaPrefix(_PREFIX_SIZE, prefix_len, prefix_k.data_ptr(), prefix_v.data_ptr(), shape[1], 0,
                       _ptr(prefix_k_scale), _ptr(prefix_v_scale), None)
    _check((_lib or load()).prefill_attn_varlen_prefix(
        *_pointers(q, k, v, cu_seqlens_q, cu_seqlens_k, cache_k, cache_v, cache_offsets, out, lse, cap, scale),
        1 if causal else 0, pre, _options(cache_k, block_table, cache_k_scale, cache_v_scale, 0, rope_theta, schedule),
        _stream_on(stream, device)))


def prefill_attn_key_weights(q, k, cu_seqlens_q, cu_seqlens_k, cache_k, cache_offsets, lse, weights, *,
                             scale: Optional[float] = None, causal: bool = True, window: int = 0, sink_tokens: int = 0,
                             prefix_len: int = 0, block_table=None, rope_theta: float = 0.0, cache_k_scale=None,
                             stream=None) -> None:
    """Adds to `weights` the softmax probability that each cached key gets from the new queries.

    weights: fp32, shape cache_k.shape[:-1].  Keys already cached are added to, the new tokens'
    keys are set.  lse is what the attention call of the same step wrote; the other arguments
    are those of that call (prefix_len: its shared prefix, for the rotary positions).
    Sequences must not share blocks of a paged cache.
    """
    if lse is None:
        raise ValueError("prefill_attn_key_weights needs lse")
    if not (-1 <= window <= _INT and -1 <= sink_tokens <= _INT and -1 <= prefix_len <= _INT):
        _int32(window=window, sink_tokens=sink_tokens, prefix_len=prefix_len)
    device, cap, _, rows = _attention_args(q, k, None, cu_seqlens_q, cu_seqlens_k, cache_k, None, cache_offsets, None, lse,
                                           block_table, cache_k_scale, cache_k_scale)
    if not (weights.dtype is _F32 and weights.shape == rows and weights.is_contiguous() and weights.get_device() == device):
        _check_tensors(device, ("weights", weights, _F32, rows))
    t, h, d = q.shape
    hk, b = k.shape[1], cache_offsets.numel()
    _check((_lib or load()).prefill_attn_key_weights(
        q.data_ptr(), k.data_ptr(), cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(), cache_k.data_ptr(),
        cache_offsets.data_ptr(), lse.data_ptr(), weights.data_ptr(), b, t, cap, h, hk, d,
        d ** -0.5 if scale is None else scale, 1 if causal else 0, sink_tokens, prefix_len,
        _options(cache_k, block_table, cache_k_scale, cache_k_scale, window, rope_theta), _stream_on(stream, device)))


def prefill_attn_evict(cache_k, cache_v, weights, lengths, kept_lengths, kept_index=None, kept_weights=None, *,
                       budget: int, sink_tokens: int = 0, recent_tokens: int = 0, block_table=None, cache_k_scale=None,
                       cache_v_scale=None, stream=None) -> None:
    """Cuts every (sequence, KV head) of the cache back to `budget` tokens by weight, in place.

    The first sink_tokens and the last recent_tokens stay, the heaviest of the rest fill the
    budget (ties: the lowest position); kept rows move to the front in their old order.
    lengths / kept_lengths int32 [num_seqs]; kept_index int32 [num_seqs, n_kv_heads, budget] or
    None; weights / kept_weights fp32 of shape cache_k.shape[:-1] (kept_weights may be weights).
    """
    if not (-1 <= budget <= _INT and -1 <= sink_tokens <= _INT and -1 <= recent_tokens <= _INT):
        _int32(budget=budget, sink_tokens=sink_tokens, recent_tokens=recent_tokens)
    device = _current_device(cache_k)
    if cache_k.dim() != 4:
        raise ValueError("caches are [num_seqs, kv_heads, cap, head_dim]")
    b, (_, hk, _, d) = lengths.numel(), cache_k.shape
    cap, _, rows = _cache_specs(device, cache_k, cache_v, b, block_table, cache_k_scale, cache_v_scale, hk, d)
    if not (weights.dtype is _F32 and weights.shape == rows and weights.is_contiguous() and weights.get_device() == device
            and lengths.dtype is _I32 and lengths.is_contiguous() and lengths.get_device() == device
            and kept_lengths.dtype is _I32 and kept_lengths.numel() == b and kept_lengths.is_contiguous()
            and kept_lengths.get_device() == device
            and (kept_index is None or kept_index.dtype is _I32 and kept_index.shape == (b, hk, budget)
                 and kept_index.is_contiguous() and kept_index.get_device() == device)
            and (kept_weights is None or kept_weights is weights
                 or kept_weights.dtype is _F32 and kept_weights.shape == rows and kept_weights.is_contiguous()
                 and kept_weights.get_device() == device)):
        _check_tensors(device, ("weights", weights, _F32, rows), ("lengths", lengths, _I32, b),
                       ("kept_lengths", kept_lengths, _I32, b), ("kept_index", kept_index, _I32, (b, hk, budget)),
                       ("kept_weights", kept_weights, _F32, rows))
    _check((_lib or load()).prefill_attn_evict(
        cache_k.data_ptr(), cache_v.data_ptr(), weights.data_ptr(), lengths.data_ptr(), kept_lengths.data_ptr(),
        _ptr(kept_index), _ptr(kept_weights), b, cap, hk, d, budget, sink_tokens, recent_tokens,
        _options(cache_k, block_table, cache_k_scale, cache_v_scale), _stream_on(stream, device)))


def _cache4(device, b, cache_k, cache_v, cache_k_params, cache_v_params, block_table, hk, d):
    """Checks a call's 4-bit cache; returns (its pa_cache4, slot capacity)."""
    if cache_k.dim() != 4 or cache_k_params.dim() != 5:
        raise ValueError("a 4-bit cache is [num_seqs, kv_heads, cap, head_dim / 2] codes, or [num_blocks, kv_heads, "
                         "block_size, head_dim / 2], with [..., head_dim / group, 2] parameters")
    shape = cache_k.shape
    n, ck_heads, rows, half = shape
    if ck_heads != hk or 2 * half != d or (block_table is None and n != b):
        raise ValueError(f"cache_k has shape {tuple(shape)}: {hk} KV heads of {d} / 2 bytes"
                         + ("" if block_table is not None else f" in {b} slots") + " are wanted")
    groups = cache_k_params.shape[3]
    if groups < 1 or d % groups:
        raise ValueError(f"cache_k_params has shape {tuple(cache_k_params.shape)}: its groups do not divide {d} channels")
    cap, params = rows, (n, hk, rows, groups, 2)
    if block_table is not None:
        if block_table.dim() != 2 or block_table.shape[0] != b:
            raise ValueError(f"block_table must be [{b}, max_blocks_per_seq]")
        cap = block_table.shape[1] * rows
        if not (block_table.dtype is _I32 and block_table.is_contiguous() and block_table.get_device() == device):
            _check_tensors(device, ("block_table", block_table, _I32, block_table.numel()))
    if not (cache_k.dtype is _U8 and cache_k.is_contiguous() and cache_k.get_device() == device
            and cache_v.dtype is _U8 and cache_v.shape == shape and cache_v.is_contiguous() and cache_v.get_device() == device
            and cache_k_params.dtype is _BF16 and cache_k_params.shape == params and cache_k_params.is_contiguous()
            and cache_k_params.get_device() == device
            and cache_v_params.dtype is _BF16 and cache_v_params.shape == params and cache_v_params.is_contiguous()
            and cache_v_params.get_device() == device):
        _check_tensors(device, ("cache_k", cache_k, _U8, shape), ("cache_v", cache_v, _U8, shape),
                       ("cache_k_params", cache_k_params, _BF16, params), ("cache_v_params", cache_v_params, _BF16, params))
    return PaCache4(_CACHE4_SIZE, d // groups, cache_k.data_ptr(), cache_v.data_ptr(), cache_k_params.data_ptr(),
                    cache_v_params.data_ptr()), cap


_U8, _CACHE4_SIZE = torch.uint8, ctypes.sizeof(PaCache4)


def prefill_attn_varlen_cache4(q, k, v, cu_seqlens_q, cu_seqlens_k, cache_k, cache_v, cache_offsets, out, lse=None, *,
                               cache_k_params, cache_v_params, scale: Optional[float] = None, causal: bool = True,
                               window: int = 0, block_table=None, rope_theta: float = 0.0, stream=None) -> None:
    """prefill_attn_varlen_ex over a cache held in 4 bits.

    cache_k/v: uint8 [num_seqs, n_kv_heads, max_cache_len, head_dim // 2], two codes to a byte (even
    channel low); cache_k_params/cache_v_params: bf16 [num_seqs, n_kv_heads, max_cache_len,
    head_dim // group, 2], scale and minimum of each group of 32, 64 or 128 channels: a channel
    stands for minimum + code * scale.  With block_table both are pools [num_blocks, n_kv_heads,
    block_size, ...].  The new tokens are attended at full precision and then stored in 4 bits.
    """
    if not -1 <= window <= _INT:
        _int32(window=window)
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q/k/v are [total_q, heads, head_dim]")
    device = _current_device(q)
    q_shape, k_shape, b = q.shape, k.shape, cache_offsets.numel()
    (t, h, d), (kt, hk, kd) = q_shape, k_shape
    if kt != t or kd != d:
        raise ValueError(f"k has shape {tuple(k_shape)}, q {tuple(q_shape)}")
    if not (q.dtype is _BF16 and k.dtype is _BF16 and q.is_contiguous() and k.is_contiguous() and k.get_device() == device
            and v.dtype is _BF16 and v.shape == k_shape and v.is_contiguous() and v.get_device() == device
            and out.dtype is _BF16 and out.shape == q_shape and out.is_contiguous() and out.get_device() == device
            and (lse is None or lse.dtype is _F32 and lse.shape == (t, h) and lse.is_contiguous()
                 and lse.get_device() == device)
            and cu_seqlens_q.dtype is _I32 and cu_seqlens_q.numel() == b + 1 and cu_seqlens_q.is_contiguous()
            and cu_seqlens_q.get_device() == device
            and cu_seqlens_k.dtype is _I32 and cu_seqlens_k.numel() == b + 1 and cu_seqlens_k.is_contiguous()
            and cu_seqlens_k.get_device() == device
            and cache_offsets.dtype is _I32 and cache_offsets.is_contiguous() and cache_offsets.get_device() == device):
        _check_tensors(device, ("q", q, _BF16, q_shape), ("k", k, _BF16, k_shape), ("v", v, _BF16, k_shape),
                       ("out", out, _BF16, q_shape), ("lse", lse, _F32, (t, h)), ("cu_seqlens_q", cu_seqlens_q, _I32, b + 1),
                       ("cu_seqlens_k", cu_seqlens_k, _I32, b + 1), ("cache_offsets", cache_offsets, _I32, b))
    cache, cap = _cache4(device, b, cache_k, cache_v, cache_k_params, cache_v_params, block_table, hk, d)
    _check((_lib or load()).prefill_attn_varlen_cache4(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(), cache,
        cache_offsets.data_ptr(), out.data_ptr(), _ptr(lse), b, t, cap, h, hk, d, d ** -0.5 if scale is None else scale,
        1 if causal else 0, _options(cache_k, block_table, None, None, window, rope_theta), _stream_on(stream, device)))


def _copy4_args(k, v, cu_seqlens, cache_k, cache_v, cache_offsets, cache_k_params, cache_v_params, block_table):
    """Checks the tensors of a write or read of a 4-bit cache; returns (device, pa_cache4, capacity)."""
    if k.dim() != 3:
        raise ValueError("k/v are [total, kv_heads, head_dim]")
    device = _current_device(k)
    shape, b = k.shape, cache_offsets.numel()
    if not (k.dtype is _BF16 and k.is_contiguous() and v.dtype is _BF16 and v.shape == shape and v.is_contiguous()
            and v.get_device() == device and cu_seqlens.dtype is _I32 and cu_seqlens.numel() == b + 1
            and cu_seqlens.is_contiguous() and cu_seqlens.get_device() == device and cache_offsets.dtype is _I32
            and cache_offsets.is_contiguous() and cache_offsets.get_device() == device):
        _check_tensors(device, ("k", k, _BF16, shape), ("v", v, _BF16, shape), ("cu_seqlens", cu_seqlens, _I32, b + 1),
                       ("cache_offsets", cache_offsets, _I32, b))
    return device, *_cache4(device, b, cache_k, cache_v, cache_k_params, cache_v_params, block_table, shape[1], shape[2])


def prefill_attn_cache4_write(k, v, cu_seqlens, cache_k, cache_v, cache_offsets, *, cache_k_params, cache_v_params,
                              block_table=None, rope_theta: float = 0.0, stream=None) -> None:
    """Quantises packed k/v [total, n_kv_heads, head_dim] (bf16) into a 4-bit cache.

    Sequence b owns rows cu_seqlens[b] .. cu_seqlens[b + 1] - 1 and its first one goes to position
    cache_offsets[b].  rope_theta > 0 rotates k to its positions first.  Caches as in
    prefill_attn_varlen_cache4.
    """
    device, cache, cap = _copy4_args(k, v, cu_seqlens, cache_k, cache_v, cache_offsets, cache_k_params, cache_v_params,
                                     block_table)
    t, hk, d = k.shape
    _check((_lib or load()).prefill_attn_cache4_write(
        k.data_ptr(), v.data_ptr(), cu_seqlens.data_ptr(), cache, cache_offsets.data_ptr(), cache_offsets.numel(), t, cap,
        hk, d, _options(cache_k, block_table, None, None, 0, rope_theta), _stream_on(stream, device)))


def prefill_attn_cache4_read(cache_k, cache_v, cu_seqlens, cache_offsets, k, v, *, cache_k_params, cache_v_params,
                             block_table=None, stream=None) -> None:
    """Reads rows of a 4-bit cache into packed k/v [total, n_kv_heads, head_dim] as bf16.

    Positions cache_offsets[b], cache_offsets[b] + 1, ... of sequence b fill rows cu_seqlens[b] ..
    cu_seqlens[b + 1] - 1: the inverse of prefill_attn_cache4_write.
    """
    device, cache, cap = _copy4_args(k, v, cu_seqlens, cache_k, cache_v, cache_offsets, cache_k_params, cache_v_params,
                                     block_table)
    t, hk, d = k.shape
    _check((_lib or load()).prefill_attn_cache4_read(
        cache, cu_seqlens.data_ptr(), cache_offsets.data_ptr(), k.data_ptr(), v.data_ptr(), cache_offsets.numel(), t, cap,
        hk, d, _options(cache_k, block_table, None, None), _stream_on(stream, device)))


def prefill_attn_varlen_noalloc(q, k, v, cu_seqlens_q, cu_seqlens_k, cache_k, cache_v, cache_offsets, out,
                                lse=None, *, scale: Optional[float] = None, causal: bool = True,
                                stream=None) -> None:
    """Same as prefill_attn_varlen, with the scheduler scratch in the library's fixed
    device array instead of an allocated workspace (see include/prefill_attn.h)."""
    args = _varlen_args(q, k, v, cu_seqlens_q, cu_seqlens_k, cache_k, cache_v, cache_offsets, out, lse,
                        scale, causal, stream)
    _check(load().prefill_attn_varlen_noalloc(*args))


def prefill_attn_varlen_validate(q, k, v, cu_seqlens_q, cu_seqlens_k, cache_k, cache_v, cache_offsets,
                                 out, lse=None, *, scale: Optional[float] = None, causal: bool = True,
                                 stream=None) -> None:
    """Strict (host-synchronising) check of the same arguments; raises on failure."""
    args = _varlen_args(q, k, v, cu_seqlens_q, cu_seqlens_k, cache_k, cache_v, cache_offsets, out, lse,
                        scale, causal, stream)
    _check(load().prefill_attn_varlen_validate(*args))


def prefill_attn_device_status(stream=None) -> int:
    """Synchronise, read and clear the device error word; returns its PA_DEVERR_* bits."""
    flags = ctypes.c_int32(0)
    st = load().prefill_attn_device_status(_stream_handle(stream), ctypes.byref(flags))
    if st not in (PA_OK, 4, 5, 6):
        _check(st)
    return flags.value


def prefill_attn_release() -> None:
    load().prefill_attn_release()


def prefill_attn_last_launch_count() -> int:
    return load().prefill_attn_last_launch_count()


def prefill_attn_last_schedule() -> int:
    """The schedule (pa_options.schedule 1, 2 or 3) the last call on this thread ran."""
    return load().prefill_attn_last_schedule()


def prefill_attn_auto_schedule(total_q: int, num_seqs: int, n_heads: int, n_kv_heads: int, kv_quant: bool,
                               num_sms: int) -> int:
    """The schedule the library picks for these sizes (host-only; -1 for rejected sizes)."""
    return load().prefill_attn_auto_schedule(total_q, num_seqs, n_heads, n_kv_heads, int(bool(kv_quant)), num_sms)
