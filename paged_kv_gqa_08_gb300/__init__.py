"""Python binding of libpagedattn: attention over a paged KV cache on GB300.

Argument marshalling only.  Each ``pa_*`` function here has the name and
argument order of the C entry point in ``include/pagedattn.h``; tensors stand
in for device pointers (``None`` for a NULL pointer) and ``stream`` defaults to
PyTorch's current stream.  Every step of the computation runs in the
library's CUDA kernels; if the library is missing, loading it raises -- there
is no other implementation to fall back to.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG_DIR, "lib", "libpagedattn.so")

PA_OK = 0
PA_ERR_NULL = 1
PA_ERR_DTYPE = 2
PA_ERR_SHAPE = 3
PA_ERR_ALIGN = 4
PA_ERR_UNSUPPORTED = 5
PA_ERR_WORKSPACE = 6
PA_ERR_CUDA = 7
PA_ERR_VALIDATION = 8
PA_ERR_CAPACITY = 9

PA_F32 = 0
PA_BF16 = 1

PA_DEVERR_BAD_SLOT = 0x1
PA_DEVERR_BAD_PAGE = 0x2
PA_DEVERR_BAD_LENGTH = 0x4
PA_DEVERR_TIMEOUT = 0x8
PA_DEVERR_NO_PAGES = 0x10


class PagedAttnError(RuntimeError):
    def __init__(self, fn: str, status: int, message: str, cuda_error: int = 0):
        self.status = status
        self.cuda_error = cuda_error
        extra = f" (cudaError {cuda_error})" if status == PA_ERR_CUDA else ""
        super().__init__(f"{fn}: status {status}: {message}{extra}")


class CacheDesc(ctypes.Structure):
    _fields_ = [("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("num_pages", ctypes.c_int64), ("dtype", ctypes.c_int32)]


def cache_desc(num_q_heads: int, num_kv_heads: int, head_dim: int, page_size: int, num_pages: int,
               dtype) -> CacheDesc:
    """Build a descriptor; ``dtype`` is torch.float32 / torch.bfloat16 or PA_F32 / PA_BF16."""
    if dtype in (torch.float32, PA_F32):
        code = PA_F32
    elif dtype in (torch.bfloat16, PA_BF16):
        code = PA_BF16
    else:
        code = int(dtype) if isinstance(dtype, int) else -1
    return CacheDesc(num_q_heads, num_kv_heads, head_dim, page_size, num_pages, code)


_lib: Optional[ctypes.CDLL] = None

_VP = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_F32 = ctypes.c_float
_DESC = ctypes.POINTER(CacheDesc)

_SIGS = {
    "pa_slot_mapping": (_I32, [_DESC, _I32, _VP, _VP, _VP, _I32, _I64, _VP, _VP, _VP]),
    "pa_kv_write": (_I32, [_DESC, _VP, _I64, _VP, _I64, _I64, _VP, _VP, _VP, _VP]),
    "pa_qk_norm_rope_kv_write": (_I32, [_DESC, _VP, _I64, _VP, _I64, _VP, _I64, _I64, _VP, _VP, _VP, _F32, _F32,
                                        _VP, _VP, _VP, _VP, _VP]),
    "pa_prefill_qk_norm_rope_kv_write": (_I32, [_DESC, _VP, _I64, _VP, _I64, _VP, _I64, _I64, _VP, _I32, _VP, _VP,
                                                _I32, _VP, _VP, _F32, _F32, _VP, _VP, _VP, _VP, _VP, _VP]),
    "pa_decode_workspace_size": (ctypes.c_size_t, [_DESC, _I32, _I32, _I32]),
    "pa_decode_plan_info": (_I32, [_DESC, _I32, _I32, _I32, ctypes.POINTER(_I32), ctypes.POINTER(_I32)]),
    "pa_decode": (_I32, [_DESC, _VP, _I32, _VP, _VP, _VP, _I32, _VP, _I32, _F32, _I32, _VP, _VP, ctypes.c_size_t,
                         _VP]),
    "pa_decode_kv_write": (_I32, [_DESC, _VP, _VP, _I64, _VP, _I64, _I32, _VP, _VP, _VP, _I32, _VP, _I32, _F32, _I32,
                                  _VP, _VP, _VP, ctypes.c_size_t, _VP]),
    "pa_decode_no_alloc": (_I32, [_DESC, _VP, _I32, _VP, _VP, _VP, _I32, _VP, _I32, _F32, _I32, _VP, _VP]),
    "pa_prefill_varlen": (_I32, [_DESC, _VP, _VP, _I32, _I32, _I64, _VP, _VP, _VP, _I32, _VP, _I32, _F32, _VP, _VP,
                                 ctypes.c_size_t, _VP]),
    "pa_prefill_step": (_I32, [_DESC, _VP, _I64, _VP, _I64, _VP, _I64, _I64, _VP, _I32, _I32, _VP, _I32, _VP, _I32,
                               _VP, _VP, _F32, _F32, _F32, _VP, _VP, _VP, _VP, _VP, _VP, _VP, ctypes.c_size_t, _VP]),
    "pa_prefill_workspace_size": (ctypes.c_size_t, [_DESC, _I32, _I32, _I64, _I32]),
    "pa_q4_row_bytes": (_I64, [_DESC, _I32]),
    "pa_kv_write_q4": (_I32, [_DESC, _I32, _VP, _I64, _VP, _I64, _I64, _VP, _VP, _VP, _VP]),
    "pa_qk_norm_rope_kv_write_q4": (_I32, [_DESC, _I32, _VP, _I64, _VP, _I64, _VP, _I64, _I64, _VP, _VP, _VP, _F32,
                                           _F32, _VP, _VP, _VP, _VP, _VP]),
    "pa_prefill_qk_norm_rope_kv_write_q4": (_I32, [_DESC, _I32, _VP, _I64, _VP, _I64, _VP, _I64, _I64, _VP, _I32, _VP,
                                                   _VP, _I32, _VP, _VP, _F32, _F32, _VP, _VP, _VP, _VP, _VP, _VP]),
    "pa_kv_read_q4": (_I32, [_DESC, _I32, _I32, _VP, _VP, _VP, _VP, _I32, _I64, _VP, _VP, _VP, _I64, _VP, _I64, _VP]),
    "pa_kv_read_q4_tables": (_I32, [_DESC, _I32, _VP, _VP, _I32, _VP, _I32, _VP]),
    "pa_decode_q4_workspace_size": (ctypes.c_size_t, [_DESC, _I32, _I32, _I32, _I32]),
    "pa_decode_q4": (_I32, [_DESC, _I32, _VP, _I32, _VP, _VP, _VP, _I32, _VP, _I32, _F32, _I32, _VP, _VP,
                            ctypes.c_size_t, _VP]),
    "pa_decode_kv_write_q4": (_I32, [_DESC, _I32, _VP, _VP, _I64, _VP, _I64, _I32, _VP, _VP, _VP, _I32, _VP, _I32,
                                     _F32, _I32, _VP, _VP, _VP, ctypes.c_size_t, _VP]),
    "pa_decode_window_workspace_size": (ctypes.c_size_t, [_DESC, _I32, _I32, _I32, _I32, _I32]),
    "pa_decode_window": (_I32, [_DESC, _I32, _I32, _VP, _I32, _VP, _VP, _VP, _I32, _VP, _I32, _F32, _I32, _VP, _VP,
                                ctypes.c_size_t, _VP]),
    "pa_decode_kv_write_window": (_I32, [_DESC, _I32, _I32, _VP, _VP, _I64, _VP, _I64, _I32, _VP, _VP, _VP, _I32, _VP,
                                         _I32, _F32, _I32, _VP, _VP, _VP, ctypes.c_size_t, _VP]),
    "pa_prefill_varlen_window": (_I32, [_DESC, _I32, _I32, _VP, _VP, _I32, _I32, _I64, _VP, _VP, _VP, _I32, _VP, _I32,
                                        _F32, _VP, _VP, ctypes.c_size_t, _VP]),
    "pa_decode_shared_prefix_workspace_size": (ctypes.c_size_t, [_DESC, _I32, _I32, _I32, _I32, _I32]),
    "pa_decode_shared_prefix": (_I32, [_DESC, _I32, _VP, _VP, _I32, _VP, _I32, _VP, _VP, _VP, _I32, _VP, _I32, _F32,
                                       _I32, _VP, _VP, ctypes.c_size_t, _VP]),
    "pa_extend_tables": (_I32, [_DESC, _I32, _VP, _VP, _VP, _I32, _VP, _VP, _I64, _VP, _VP, _VP, _VP, _VP, _VP, _VP]),
    "pa_share_pages": (_I32, [_DESC, _I32, _VP, _VP, _VP, _I32, _VP, _VP]),
    "pa_release_pages": (_I32, [_DESC, _I32, _VP, _VP, _VP, _I32, _VP, _VP, _VP, _VP, _VP]),
    "pa_release_window_pages": (_I32, [_DESC, _I32, _I32, _I32, _VP, _VP, _I32, _VP, _VP, _VP, _VP, _VP]),
    "pa_validate_metadata": (_I32, [_DESC, _I32, _VP, _VP, _VP, _I32, _I32, _VP, _VP]),
    "pa_selftest_bounded_wait": (_I32, [_I32, _VP]),
    "pa_read_device_errors": (_I32, [ctypes.POINTER(ctypes.c_uint32), _I32]),
    "pa_last_cuda_error": (_I32, []),
    "pa_status_string": (ctypes.c_char_p, [_I32]),
    "pa_version": (_I32, []),
    "pa_bm_create": (_I32, [_I64, _I32, ctypes.POINTER(_VP)]),
    "pa_bm_destroy": (None, [_VP]),
    "pa_bm_can_allocate": (_I32, [_VP, _VP, _I64, ctypes.POINTER(_I64)]),
    "pa_bm_allocate": (_I32, [_VP, _I64, _VP, _I64, ctypes.POINTER(_I64)]),
    "pa_bm_append_token": (_I32, [_VP, _I64, _I32]),
    "pa_bm_hash_blocks": (_I32, [_VP, _I64, _I64]),
    "pa_bm_free": (_I32, [_VP, _I64]),
    "pa_bm_block_tables": (_I32, [_VP, _VP, _I32, _I32, _I32, _VP, _VP]),
    "pa_bm_slot_mapping": (_I32, [_VP, _VP, _I32, _VP, _VP]),
    "pa_bm_query": (_I32, [_VP, ctypes.POINTER(_I64), ctypes.POINTER(_I64), ctypes.POINTER(_I64)]),
    "pa_bm_block_ref_count": (_I32, [_VP, _I32, ctypes.POINTER(_I32)]),
    "pa_bm_seq_info": (_I32, [_VP, _I64, ctypes.POINTER(_I64), ctypes.POINTER(_I64), ctypes.POINTER(_I32)]),
}


def load_library(path: Optional[str] = None) -> ctypes.CDLL:
    """Load libpagedattn.so (built by ``paged_kv_gqa_08_gb300.build``)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise ImportError(f"libpagedattn.so not found at {p}; build it with "
                          "`python -m paged_kv_gqa_08_gb300.build`")
    lib = ctypes.CDLL(p)
    for name, (res, args) in _SIGS.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    if path is None:
        _lib = lib
    return lib


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, torch.Tensor):
        return t.data_ptr() if t.numel() > 0 else None
    return int(t)


def _at(t) -> Optional[int]:
    """_ptr for the short calls: a tensor's address, whatever its size (the library looks at the sizes it is given)."""
    try:
        return t.data_ptr()
    except AttributeError:
        return None if t is None else int(t)


_Tensor, _uint8 = torch.Tensor, torch.uint8

# The current device's index and its current stream's handle, as torch.cuda.current_device() and
# current_stream().cuda_stream give them, without their layers of checks: those took 4 us of a call's 14.
_current_device = None
_raw_stream = None


def _find_cuda() -> bool:
    """Whether there is a CUDA device; sets up the two lookups above once there is."""
    global _current_device, _raw_stream
    if not torch.cuda.is_available():
        return False
    torch.cuda.init()
    _raw_stream = torch._C._cuda_getCurrentRawStream
    _current_device = torch._C._cuda_getDevice
    return True


def _stream(stream) -> Optional[int]:
    if stream is None:
        if _current_device is None and not _find_cuda():
            return None
        return _raw_stream(_current_device())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _check(fn: str, status: int) -> None:
    if status != PA_OK:
        lib = load_library()
        msg = lib.pa_status_string(status).decode()
        raise PagedAttnError(fn, status, msg, lib.pa_last_cuda_error())


def pa_slot_mapping(desc, batch, cu_seqlens_q, context_lens, block_tables, max_pages_per_seq, num_tokens,
                    positions, slot_mapping, stream=None):
    lib = load_library()
    _check("pa_slot_mapping", lib.pa_slot_mapping(
        ctypes.byref(desc), batch, _ptr(cu_seqlens_q), _ptr(context_lens), _ptr(block_tables),
        max_pages_per_seq, num_tokens, _ptr(positions), _ptr(slot_mapping), _stream(stream)))


def pa_kv_write(desc, k, k_row_stride, v, v_row_stride, num_tokens, slot_mapping, k_cache, v_cache, stream=None):
    lib = load_library()
    _check("pa_kv_write", lib.pa_kv_write(
        ctypes.byref(desc), _ptr(k), k_row_stride, _ptr(v), v_row_stride, num_tokens, _ptr(slot_mapping),
        _ptr(k_cache), _ptr(v_cache), _stream(stream)))


def pa_qk_norm_rope_kv_write(desc, q, q_row_stride, k, k_row_stride, v, v_row_stride, num_tokens, positions,
                             q_norm_w, k_norm_w, eps, rope_theta, slot_mapping, q_out, k_cache, v_cache,
                             stream=None):
    lib = load_library()
    _check("pa_qk_norm_rope_kv_write", lib.pa_qk_norm_rope_kv_write(
        ctypes.byref(desc), _ptr(q), q_row_stride, _ptr(k), k_row_stride, _ptr(v), v_row_stride, num_tokens,
        _ptr(positions), _ptr(q_norm_w), _ptr(k_norm_w), eps, rope_theta, _ptr(slot_mapping), _ptr(q_out),
        _ptr(k_cache), _ptr(v_cache), _stream(stream)))


def pa_prefill_qk_norm_rope_kv_write(desc, q, q_row_stride, k, k_row_stride, v, v_row_stride, num_tokens,
                                     cu_seqlens_q, batch, context_lens, block_tables, max_pages_per_seq, q_norm_w,
                                     k_norm_w, eps, rope_theta, q_out, k_cache, v_cache, positions_out=None,
                                     slot_mapping_out=None, stream=None):
    lib = load_library()
    _check("pa_prefill_qk_norm_rope_kv_write", lib.pa_prefill_qk_norm_rope_kv_write(
        ctypes.byref(desc), _ptr(q), q_row_stride, _ptr(k), k_row_stride, _ptr(v), v_row_stride, num_tokens,
        _ptr(cu_seqlens_q), batch, _ptr(context_lens), _ptr(block_tables), max_pages_per_seq, _ptr(q_norm_w),
        _ptr(k_norm_w), eps, rope_theta, _ptr(q_out), _ptr(k_cache), _ptr(v_cache), _ptr(positions_out),
        _ptr(slot_mapping_out), _stream(stream)))


def pa_decode_workspace_size(desc, batch, max_context_len, max_ctas=0) -> int:
    return int(load_library().pa_decode_workspace_size(ctypes.byref(desc), batch, max_context_len, max_ctas))


def pa_decode_plan_info(desc, batch, max_context_len, max_ctas=0):
    """(num_partitions, tokens_per_chunk) pa_decode would use on the current device."""
    lib = load_library()
    n = _I32(0)
    t = _I32(0)
    _check("pa_decode_plan_info", lib.pa_decode_plan_info(ctypes.byref(desc), batch, max_context_len, max_ctas,
                                                          ctypes.byref(n), ctypes.byref(t)))
    return int(n.value), int(t.value)


def pa_decode(desc, q, batch, k_cache, v_cache, block_tables, max_pages_per_seq, context_lens, max_context_len,
              scale, max_ctas, out, workspace, workspace_bytes=None, stream=None):
    lib = load_library()
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("pa_decode", lib.pa_decode(
        ctypes.byref(desc), _ptr(q), batch, _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), max_pages_per_seq,
        _ptr(context_lens), max_context_len, scale, max_ctas, _ptr(out), _ptr(workspace), workspace_bytes,
        _stream(stream)))


def pa_decode_kv_write(desc, q, k_new, k_row_stride, v_new, v_row_stride, batch, k_cache, v_cache, block_tables,
                       max_pages_per_seq, context_lens, max_context_len, scale, max_ctas, slot_mapping, out, workspace,
                       workspace_bytes=None, stream=None):
    lib = load_library()
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("pa_decode_kv_write", lib.pa_decode_kv_write(
        ctypes.byref(desc), _ptr(q), _ptr(k_new), k_row_stride, _ptr(v_new), v_row_stride, batch, _ptr(k_cache),
        _ptr(v_cache), _ptr(block_tables), max_pages_per_seq, _ptr(context_lens), max_context_len, scale, max_ctas,
        _ptr(slot_mapping), _ptr(out), _ptr(workspace), workspace_bytes, _stream(stream)))


def pa_decode_no_alloc(desc, q, batch, k_cache, v_cache, block_tables, max_pages_per_seq, context_lens,
                       max_context_len, scale, max_ctas, out, stream=None):
    """pa_decode with the library's fixed 16 MiB scratch instead of a caller workspace."""
    lib = load_library()
    _check("pa_decode_no_alloc", lib.pa_decode_no_alloc(
        ctypes.byref(desc), _ptr(q), batch, _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), max_pages_per_seq,
        _ptr(context_lens), max_context_len, scale, max_ctas, _ptr(out), _stream(stream)))


def pa_prefill_varlen(desc, q, cu_seqlens_q, batch, max_seqlen_q, num_tokens, k_cache, v_cache, block_tables,
                      max_pages_per_seq, context_lens, max_context_len, scale, out, workspace=None,
                      workspace_bytes=None, stream=None):
    lib = load_library()
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("pa_prefill_varlen", lib.pa_prefill_varlen(
        ctypes.byref(desc), _ptr(q), _ptr(cu_seqlens_q), batch, max_seqlen_q, num_tokens, _ptr(k_cache),
        _ptr(v_cache), _ptr(block_tables), max_pages_per_seq, _ptr(context_lens), max_context_len, scale,
        _ptr(out), _ptr(workspace), workspace_bytes, _stream(stream)))


def pa_prefill_step(desc, q, q_row_stride, k, k_row_stride, v, v_row_stride, num_tokens, cu_seqlens_q, batch,
                    max_seqlen_q, context_lens, max_context_len, block_tables, max_pages_per_seq, q_norm_w, k_norm_w,
                    eps, rope_theta, scale, q_out, k_cache, v_cache, positions_out, slot_mapping_out, out,
                    workspace=None, workspace_bytes=None, stream=None):
    lib = load_library()
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("pa_prefill_step", lib.pa_prefill_step(
        ctypes.byref(desc), _ptr(q), q_row_stride, _ptr(k), k_row_stride, _ptr(v), v_row_stride, num_tokens,
        _ptr(cu_seqlens_q), batch, max_seqlen_q, _ptr(context_lens), max_context_len, _ptr(block_tables),
        max_pages_per_seq, _ptr(q_norm_w), _ptr(k_norm_w), eps, rope_theta, scale, _ptr(q_out), _ptr(k_cache),
        _ptr(v_cache), _ptr(positions_out), _ptr(slot_mapping_out), _ptr(out), _ptr(workspace), workspace_bytes,
        _stream(stream)))


def pa_prefill_workspace_size(desc, batch, max_seqlen_q, num_tokens, max_context_len) -> int:
    return int(load_library().pa_prefill_workspace_size(ctypes.byref(desc), batch, max_seqlen_q, num_tokens,
                                                        max_context_len))


def pa_q4_row_bytes(desc, group_size) -> int:
    """Bytes of one token's row of a 4-bit K or V cache (0: not supported)."""
    return int(load_library().pa_q4_row_bytes(desc, group_size))


def _q4_cache_shapes(fn, desc, group_size, k_cache, v_cache):
    """A 4-bit cache given as a tensor is contiguous uint8 and holds every row of the descriptor: a cache of the dtype's
    rows, or one allocated for another group size, is refused here."""
    need = desc.num_pages * desc.page_size * load_library().pa_q4_row_bytes(desc, group_size)
    for t in (k_cache, v_cache):
        if not isinstance(t, torch.Tensor):
            continue
        if t.dtype is not torch.uint8:
            raise PagedAttnError(fn, PA_ERR_DTYPE, f"a 4-bit cache is a uint8 tensor, not {t.dtype}")
        if t.numel() < need or not t.is_contiguous():
            raise PagedAttnError(fn, PA_ERR_SHAPE, f"a 4-bit cache is contiguous and has at least {need} bytes")


def _q4_caches(fn, desc, group_size, k_cache, v_cache):
    """Those checks, and that a cache given as a tensor is on the current device."""
    _q4_cache_shapes(fn, desc, group_size, k_cache, v_cache)
    for t in (k_cache, v_cache):
        if isinstance(t, torch.Tensor) and ((_current_device is None and not _find_cuda()) or
                                            t.get_device() != _current_device()):
            raise PagedAttnError(fn, PA_ERR_UNSUPPORTED, f"the cache is on {t.device}, not on the current CUDA device")


def _q4_args(fn, desc, group_size, k_cache, v_cache, stream, *tensors):
    """The addresses of ``tensors`` and of the checked caches, and the stream: what every call over a 4-bit cache
    passes on.  The calls are short, so the usual case (tensors, the current stream) takes the fewest steps."""
    at = [t.data_ptr() if t.__class__ is _Tensor else _at(t) for t in tensors]
    if k_cache.__class__ is _Tensor and v_cache.__class__ is _Tensor and _current_device is not None:
        device = _current_device()
        need = desc.num_pages * desc.page_size * _lib.pa_q4_row_bytes(desc, group_size)
        if (k_cache.dtype is _uint8 and k_cache.numel() >= need and k_cache.is_contiguous()
                and k_cache.get_device() == device and v_cache.dtype is _uint8 and v_cache.numel() >= need
                and v_cache.is_contiguous() and v_cache.get_device() == device):
            return at, k_cache.data_ptr(), v_cache.data_ptr(), (_raw_stream(device) if stream is None
                                                                else _stream(stream))
    _q4_caches(fn, desc, group_size, k_cache, v_cache)
    return at, _at(k_cache), _at(v_cache), _stream(stream)


def pa_kv_write_q4(desc, group_size, k, k_row_stride, v, v_row_stride, num_tokens, slot_mapping, k_cache, v_cache,
                   stream=None):
    lib = load_library()
    (k, v, slots), kc, vc, st = _q4_args("pa_kv_write_q4", desc, group_size, k_cache, v_cache, stream, k, v,
                                         slot_mapping)
    _check("pa_kv_write_q4", lib.pa_kv_write_q4(desc, group_size, k, k_row_stride, v, v_row_stride, num_tokens, slots,
                                                kc, vc, st))


def pa_qk_norm_rope_kv_write_q4(desc, group_size, q, q_row_stride, k, k_row_stride, v, v_row_stride, num_tokens,
                                positions, q_norm_w, k_norm_w, eps, rope_theta, slot_mapping, q_out, k_cache, v_cache,
                                stream=None):
    lib = load_library()
    (q, k, v, pos, wq, wk, slots, qo), kc, vc, st = _q4_args(
        "pa_qk_norm_rope_kv_write_q4", desc, group_size, k_cache, v_cache, stream, q, k, v, positions, q_norm_w,
        k_norm_w, slot_mapping, q_out)
    _check("pa_qk_norm_rope_kv_write_q4", lib.pa_qk_norm_rope_kv_write_q4(
        desc, group_size, q, q_row_stride, k, k_row_stride, v, v_row_stride, num_tokens, pos, wq, wk, eps, rope_theta,
        slots, qo, kc, vc, st))


def pa_prefill_qk_norm_rope_kv_write_q4(desc, group_size, q, q_row_stride, k, k_row_stride, v, v_row_stride,
                                        num_tokens, cu_seqlens_q, batch, context_lens, block_tables,
                                        max_pages_per_seq, q_norm_w, k_norm_w, eps, rope_theta, q_out, k_cache,
                                        v_cache, positions_out=None, slot_mapping_out=None, stream=None):
    lib = load_library()
    (q, k, v, cu, ctx, bt, wq, wk, qo, pos, slots), kc, vc, st = _q4_args(
        "pa_prefill_qk_norm_rope_kv_write_q4", desc, group_size, k_cache, v_cache, stream, q, k, v, cu_seqlens_q,
        context_lens, block_tables, q_norm_w, k_norm_w, q_out, positions_out, slot_mapping_out)
    _check("pa_prefill_qk_norm_rope_kv_write_q4", lib.pa_prefill_qk_norm_rope_kv_write_q4(
        desc, group_size, q, q_row_stride, k, k_row_stride, v, v_row_stride, num_tokens, cu, batch, ctx, bt,
        max_pages_per_seq, wq, wk, eps, rope_theta, qo, kc, vc, pos, slots, st))


def pa_kv_read_q4(desc, group_size, batch, cu_rows, starts, context_lens, block_tables, max_pages_per_seq, num_rows,
                  k_cache, v_cache, k_out, k_row_stride, v_out, v_row_stride, stream=None):
    """Read tokens of a 4-bit cache back as rows of the descriptor's dtype; ``starts`` may be None (token 0)."""
    lib = load_library()
    (cu, starts, ctx, bt, ko, vo), kc, vc, st = _q4_args(
        "pa_kv_read_q4", desc, group_size, k_cache, v_cache, stream, cu_rows, starts, context_lens, block_tables,
        k_out, v_out)
    _check("pa_kv_read_q4", lib.pa_kv_read_q4(
        desc, group_size, batch, cu, starts, ctx, bt, max_pages_per_seq, num_rows, kc, vc, ko, k_row_stride, vo,
        v_row_stride, st))


def pa_kv_read_q4_tables(desc, batch, cu_rows, block_tables, max_pages_per_seq, tables_out, max_pages_out,
                         stream=None):
    """Block tables of the paged cache that a ``pa_kv_read_q4`` of whole pages filled: -1 where no page was read."""
    _check("pa_kv_read_q4_tables", load_library().pa_kv_read_q4_tables(
        desc, batch, _at(cu_rows), _at(block_tables), max_pages_per_seq, _at(tables_out), max_pages_out,
        _stream(stream)))


def pa_decode_q4_workspace_size(desc, group_size, batch, max_context_len, max_ctas=0) -> int:
    return int(load_library().pa_decode_q4_workspace_size(desc, group_size, batch, max_context_len,
                                                          max_ctas))


def pa_decode_q4(desc, group_size, q, batch, k_cache, v_cache, block_tables, max_pages_per_seq, context_lens,
                 max_context_len, scale, max_ctas, out, workspace, workspace_bytes=None, stream=None):
    lib = load_library()
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    (q, bt, ctx, out, ws), kc, vc, st = _q4_args("pa_decode_q4", desc, group_size, k_cache, v_cache, stream, q,
                                                 block_tables, context_lens, out, workspace)
    _check("pa_decode_q4", lib.pa_decode_q4(
        desc, group_size, q, batch, kc, vc, bt, max_pages_per_seq, ctx, max_context_len, scale, max_ctas, out, ws,
        workspace_bytes, st))


def pa_decode_kv_write_q4(desc, group_size, q, k_new, k_row_stride, v_new, v_row_stride, batch, k_cache, v_cache,
                          block_tables, max_pages_per_seq, context_lens, max_context_len, scale, max_ctas,
                          slot_mapping, out, workspace, workspace_bytes=None, stream=None):
    lib = load_library()
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    (q, k, v, bt, ctx, slots, out, ws), kc, vc, st = _q4_args(
        "pa_decode_kv_write_q4", desc, group_size, k_cache, v_cache, stream, q, k_new, v_new, block_tables,
        context_lens, slot_mapping, out, workspace)
    _check("pa_decode_kv_write_q4", lib.pa_decode_kv_write_q4(
        desc, group_size, q, k, k_row_stride, v, v_row_stride, batch, kc, vc, bt, max_pages_per_seq, ctx,
        max_context_len, scale, max_ctas, slots, out, ws, workspace_bytes, st))


def _addresses(*tensors):
    """The addresses of ``tensors``: the calls are short, so the usual case takes the fewest steps."""
    return [t.data_ptr() if t.__class__ is _Tensor else _at(t) for t in tensors]


def _bytes_of(workspace, workspace_bytes):
    if workspace_bytes is None:
        return workspace.numel() * workspace.element_size() if workspace is not None else 0
    return workspace_bytes


def pa_decode_window_workspace_size(desc, window, num_sinks, batch, max_context_len, max_ctas=0) -> int:
    return int(load_library().pa_decode_window_workspace_size(desc, window, num_sinks, batch, max_context_len,
                                                              max_ctas))


def pa_decode_window(desc, window, num_sinks, q, batch, k_cache, v_cache, block_tables, max_pages_per_seq,
                     context_lens, max_context_len, scale, max_ctas, out, workspace, workspace_bytes=None,
                     stream=None):
    q, kc, vc, bt, ctx, o, ws = _addresses(q, k_cache, v_cache, block_tables, context_lens, out, workspace)
    _check("pa_decode_window", load_library().pa_decode_window(
        desc, window, num_sinks, q, batch, kc, vc, bt, max_pages_per_seq, ctx, max_context_len, scale, max_ctas, o, ws,
        _bytes_of(workspace, workspace_bytes), _stream(stream)))


def pa_decode_kv_write_window(desc, window, num_sinks, q, k_new, k_row_stride, v_new, v_row_stride, batch, k_cache,
                              v_cache, block_tables, max_pages_per_seq, context_lens, max_context_len, scale, max_ctas,
                              slot_mapping, out, workspace, workspace_bytes=None, stream=None):
    q, k, v, kc, vc, bt, ctx, slots, o, ws = _addresses(q, k_new, v_new, k_cache, v_cache, block_tables, context_lens,
                                                        slot_mapping, out, workspace)
    _check("pa_decode_kv_write_window", load_library().pa_decode_kv_write_window(
        desc, window, num_sinks, q, k, k_row_stride, v, v_row_stride, batch, kc, vc, bt, max_pages_per_seq, ctx,
        max_context_len, scale, max_ctas, slots, o, ws, _bytes_of(workspace, workspace_bytes), _stream(stream)))


def pa_prefill_varlen_window(desc, window, num_sinks, q, cu_seqlens_q, batch, max_seqlen_q, num_tokens, k_cache,
                             v_cache, block_tables, max_pages_per_seq, context_lens, max_context_len, scale, out,
                             workspace=None, workspace_bytes=None, stream=None):
    q, cu, kc, vc, bt, ctx, o, ws = _addresses(q, cu_seqlens_q, k_cache, v_cache, block_tables, context_lens, out,
                                               workspace)
    _check("pa_prefill_varlen_window", load_library().pa_prefill_varlen_window(
        desc, window, num_sinks, q, cu, batch, max_seqlen_q, num_tokens, kc, vc, bt, max_pages_per_seq, ctx,
        max_context_len, scale, o, ws, _bytes_of(workspace, workspace_bytes), _stream(stream)))


def pa_decode_shared_prefix_workspace_size(desc, num_groups, batch, max_prefix_len, max_context_len,
                                           max_ctas=0) -> int:
    return int(load_library().pa_decode_shared_prefix_workspace_size(desc, num_groups, batch, max_prefix_len,
                                                                     max_context_len, max_ctas))


def pa_decode_shared_prefix(desc, num_groups, cu_groups, prefix_lens, max_prefix_len, q, batch, k_cache, v_cache,
                            block_tables, max_pages_per_seq, context_lens, max_context_len, scale, max_ctas, out,
                            workspace, workspace_bytes=None, stream=None):
    cu, pre, q, kc, vc, bt, ctx, o, ws = _addresses(cu_groups, prefix_lens, q, k_cache, v_cache, block_tables,
                                                    context_lens, out, workspace)
    _check("pa_decode_shared_prefix", load_library().pa_decode_shared_prefix(
        desc, num_groups, cu, pre, max_prefix_len, q, batch, kc, vc, bt, max_pages_per_seq, ctx, max_context_len, scale,
        max_ctas, o, ws, _bytes_of(workspace, workspace_bytes), _stream(stream)))


def pa_extend_tables(desc, batch, new_tokens, context_lens, block_tables, max_pages_per_seq, free_pages, pool_state,
                     max_tokens, cu_seqlens_q, context_lens_out, positions, slot_mapping, ref_counts, pool_state_out,
                     stream=None):
    new, ctx, bt, ring, pool, cu, ctx_out, pos, slots, refs, pool_out = _addresses(
        new_tokens, context_lens, block_tables, free_pages, pool_state, cu_seqlens_q, context_lens_out, positions,
        slot_mapping, ref_counts, pool_state_out)
    _check("pa_extend_tables", load_library().pa_extend_tables(
        desc, batch, new, ctx, bt, max_pages_per_seq, ring, pool, max_tokens, cu, ctx_out, pos, slots, refs, pool_out,
        _stream(stream)))


def pa_share_pages(desc, batch, parents, num_shared_pages, block_tables, max_pages_per_seq, ref_counts, stream=None):
    _check("pa_share_pages", load_library().pa_share_pages(
        desc, batch, _at(parents), _at(num_shared_pages), _at(block_tables), max_pages_per_seq, _at(ref_counts),
        _stream(stream)))


def pa_release_pages(desc, batch, first_pages, end_pages, block_tables, max_pages_per_seq, ref_counts, free_pages,
                     pool_state, pool_state_out, stream=None):
    first, end, bt, refs, ring, pool, pool_out = _addresses(first_pages, end_pages, block_tables, ref_counts, free_pages,
                                                            pool_state, pool_state_out)
    _check("pa_release_pages", load_library().pa_release_pages(
        desc, batch, first, end, bt, max_pages_per_seq, refs, ring, pool, pool_out, _stream(stream)))


def pa_release_window_pages(desc, window, num_sinks, batch, context_lens, block_tables, max_pages_per_seq, ref_counts,
                            free_pages, pool_state, pool_state_out, stream=None):
    _check("pa_release_window_pages", load_library().pa_release_window_pages(
        desc, window, num_sinks, batch, _at(context_lens), _at(block_tables), max_pages_per_seq, _at(ref_counts),
        _at(free_pages), _at(pool_state), _at(pool_state_out), _stream(stream)))


def pa_validate_metadata(desc, batch, cu_seqlens_q, context_lens, block_tables, max_pages_per_seq,
                         max_context_len, error_count, stream=None):
    lib = load_library()
    _check("pa_validate_metadata", lib.pa_validate_metadata(
        ctypes.byref(desc), batch, _ptr(cu_seqlens_q), _ptr(context_lens), _ptr(block_tables), max_pages_per_seq,
        max_context_len, _ptr(error_count), _stream(stream)))


def pa_selftest_bounded_wait(timeout_ms: int, stream=None):
    _check("pa_selftest_bounded_wait", load_library().pa_selftest_bounded_wait(timeout_ms, _stream(stream)))


def pa_read_device_errors(reset: bool = False) -> int:
    lib = load_library()
    flags = ctypes.c_uint32(0)
    _check("pa_read_device_errors", lib.pa_read_device_errors(ctypes.byref(flags), 1 if reset else 0))
    return int(flags.value)


def pa_status_string(status: int) -> str:
    return load_library().pa_status_string(status).decode()


def pa_version() -> int:
    return int(load_library().pa_version())
