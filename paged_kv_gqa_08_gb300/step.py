"""One attention-layer step over a paged KV cache, through the C ABI.

The order is the nano-vLLM learning note's (Qwen3Attention.forward and
Attention.forward listings): positions and slots of the step's new tokens,
optional per-head q/k RMSNorm + rotary, the KV write, then decode or
chunked-prefill attention over the cache.  This module only allocates buffers
and sequences calls; every value is computed by libpagedattn's kernels.

Buffers allocated with a ``group_size`` step over a 4-bit cache: the writes
quantise, decode attends to the codes, and prefill reads the contexts back into
a staging cache of the descriptor's dtype and attends to that.

A step with a ``window`` attends to the last ``window`` tokens and the first
``num_sinks``; a decode step with ``cu_groups`` reads the prefix that the requests
of a group share once for all of them.
"""
from __future__ import annotations

import dataclasses
import math
from typing import Optional

import torch

from . import (PA_ERR_ALIGN, PA_ERR_NULL, PA_ERR_SHAPE, PA_ERR_UNSUPPORTED, PA_ERR_WORKSPACE, PagedAttnError, _at,
               _q4_cache_shapes, cache_desc, pa_decode, pa_decode_q4, pa_decode_q4_workspace_size, pa_decode_shared_prefix,
               pa_decode_shared_prefix_workspace_size, pa_decode_window, pa_decode_window_workspace_size,
               pa_decode_workspace_size, pa_kv_read_q4, pa_kv_read_q4_tables, pa_kv_write, pa_kv_write_q4,
               pa_prefill_qk_norm_rope_kv_write, pa_prefill_qk_norm_rope_kv_write_q4, pa_prefill_step,
               pa_prefill_varlen, pa_prefill_varlen_window, pa_prefill_workspace_size, pa_slot_mapping)


@dataclasses.dataclass
class Staging:
    """Where a prefill step over a 4-bit cache reads the contexts back to: a paged cache of the descriptor's dtype
    in which request b has the ``max_pages`` pages from ``b * max_pages`` on.  Each step writes its own block tables:
    they leave out the pages that its read-back could not fill."""
    desc: object                       # the staging cache's descriptor
    max_pages: int
    cu_rows: torch.Tensor              # int32 [batch + 1]
    block_tables: torch.Tensor         # int32 [batch, max_pages]
    k: torch.Tensor                    # [batch * max_pages, page_size, Hkv, hd]
    v: torch.Tensor


@dataclasses.dataclass
class StepBuffers:
    positions: torch.Tensor            # int32 [N]
    slots: torch.Tensor                # int64 [N]
    out: torch.Tensor                  # [N, Hq, hd]
    q_out: Optional[torch.Tensor]      # [N, Hq, hd] normed + rotated q (when norm weights are used)
    workspace: Optional[torch.Tensor]  # decode split-KV / planned-prefill workspace (bytes)
    max_ctas: int = 0
    group_size: int = 0                # dims that share a scale in a 4-bit cache; 0: a cache of the dtype's rows
    staging: Optional[Staging] = None  # prefill over a 4-bit cache


def torch_dtype(desc) -> torch.dtype:
    return torch.float32 if desc.dtype == 0 else torch.bfloat16


def alloc_step_buffers(desc, kind: str, num_tokens: int, batch: int, max_context_len: int, device,
                       norm: bool = False, max_ctas: int = 0, max_seqlen_q: Optional[int] = None,
                       plan_prefill: bool = True, group_size: int = 0, window: int = 0, num_sinks: int = 0,
                       num_groups: int = 0, max_prefix_len: int = 0) -> StepBuffers:
    """Buffers of one step.  A prefill step gets the planned-launch workspace
    unless ``plan_prefill`` is False (or the shape is never planned); it is
    sized for chunks up to ``max_seqlen_q`` tokens (default: ``num_tokens``).
    ``group_size`` (32, 64 or 128) is that of a 4-bit cache; a prefill step over
    one gets a staging cache for ``batch`` contexts of ``max_context_len``.
    ``window`` and ``num_sinks``, or ``num_groups`` and ``max_prefix_len``, are those
    that a decode step will be run with."""
    dt = torch_dtype(desc)
    n = max(num_tokens, 1)
    positions = torch.empty(n, dtype=torch.int32, device=device)
    slots = torch.empty(n, dtype=torch.int64, device=device)
    out = torch.empty(n, desc.num_q_heads, desc.head_dim, dtype=dt, device=device)
    q_out = torch.empty_like(out) if norm else None
    ws = None
    if kind == "decode":
        if group_size:
            fn = "pa_decode_q4_workspace_size"
            nbytes = pa_decode_q4_workspace_size(desc, group_size, batch, max_context_len, max_ctas)
        elif window:
            fn = "pa_decode_window_workspace_size"
            nbytes = pa_decode_window_workspace_size(desc, window, num_sinks, batch, max_context_len, max_ctas)
        elif num_groups:
            fn = "pa_decode_shared_prefix_workspace_size"
            nbytes = pa_decode_shared_prefix_workspace_size(desc, num_groups, batch, max_prefix_len, max_context_len,
                                                            max_ctas)
        else:
            fn = "pa_decode_workspace_size"
            nbytes = pa_decode_workspace_size(desc, batch, max_context_len, max_ctas)
        if nbytes == 0:
            raise RuntimeError(fn + " returned 0 (unsupported shape or no device)")
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    elif plan_prefill and num_tokens > 0:
        nbytes = pa_prefill_workspace_size(desc, batch, max_seqlen_q or num_tokens, num_tokens, max_context_len)
        if nbytes:
            ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    staging = None
    if group_size and kind != "decode":
        P = desc.page_size
        max_pages = max(-(-max_context_len // P), 1)
        pages = max(batch, 1) * max_pages
        if pages * P >= 2 ** 31:
            raise ValueError("the staged contexts have more than 2^31 - 1 rows")
        shape = (pages, P, desc.num_kv_heads, desc.head_dim)
        staging = Staging(cache_desc(desc.num_q_heads, desc.num_kv_heads, desc.head_dim, P, pages, dt), max_pages,
                          torch.arange(0, pages * P + 1, max_pages * P, dtype=torch.int32, device=device),
                          torch.empty(max(batch, 1), max_pages, dtype=torch.int32, device=device),
                          torch.empty(shape, dtype=dt, device=device), torch.empty(shape, dtype=dt, device=device))
    return StepBuffers(positions, slots, out, q_out, ws, max_ctas, group_size, staging)


def write_rows(desc, k_rows, v_rows, cu_rows, lens, block_tables, max_pages_per_seq, bufs_positions, bufs_slots,
               k_cache, v_cache, stream=None, group_size: int = 0):
    """Store already-computed K/V rows (the last ``cu_rows`` segment of each of
    ``lens[b]`` tokens) into their slots: slot mapping then KV write.
    ``group_size``: that of a 4-bit cache."""
    n = k_rows.shape[0]
    batch = lens.shape[0]
    if n == 0:
        return
    pa_slot_mapping(desc, batch, cu_rows, lens, block_tables, max_pages_per_seq, n, bufs_positions, bufs_slots,
                    stream)
    row = desc.num_kv_heads * desc.head_dim
    if group_size:
        pa_kv_write_q4(desc, group_size, k_rows, row, v_rows, row, n, bufs_slots, k_cache, v_cache, stream)
        return
    pa_kv_write(desc, k_rows, row, v_rows, row, n, bufs_slots, k_cache, v_cache, stream)


def run_step(desc, kind: str, bufs: StepBuffers, q, k, v, cu_seqlens_q, context_lens, block_tables,
             k_cache, v_cache, scale: float, max_pages_per_seq: int, max_context_len: int, max_seqlen_q: int,
             q_norm_w=None, k_norm_w=None, eps: float = 0.0, rope_theta: float = 0.0, stream=None, window: int = 0,
             num_sinks: int = 0, cu_groups=None, prefix_lens=None, max_prefix_len: int = 0):
    """Run one step; returns ``bufs.out`` (the attention output of the new tokens).  A step beyond its buffers is a
    ``ValueError``; over a 4-bit cache, with a window and with groups whatever is refused is refused before anything is
    enqueued.

    ``window`` > 0: the tokens attended to are those of ``pa_decode_window`` and ``pa_prefill_varlen_window``.
    ``cu_groups`` and ``prefix_lens`` (up to ``max_prefix_len``): the groups of ``pa_decode_shared_prefix``, for decode
    steps.  One or the other, and not over a 4-bit cache."""
    n = q.shape[0]
    batch = context_lens.shape[0]
    for t in (bufs.positions, bufs.slots, bufs.out, bufs.q_out if q_norm_w is not None else None):
        if t is not None and t.shape[0] < n:
            raise ValueError(f"a step of {n} tokens in buffers for {t.shape[0]}")
    if window or cu_groups is not None:
        return _run_step_range(desc, kind, bufs, q, k, v, cu_seqlens_q, context_lens, block_tables, k_cache, v_cache,
                               scale, max_pages_per_seq, max_context_len, max_seqlen_q, q_norm_w, k_norm_w, eps,
                               rope_theta, stream, window, num_sinks, cu_groups, prefix_lens, max_prefix_len)
    if bufs.group_size:
        return _run_step_q4(desc, kind, bufs, q, k, v, cu_seqlens_q, context_lens, block_tables, k_cache, v_cache,
                            scale, max_pages_per_seq, max_context_len, max_seqlen_q, q_norm_w, k_norm_w, eps,
                            rope_theta, stream)
    if kind != "decode":
        # the write part and the attention in one call, whose attention planner
        # runs beside the write kernel
        pa_prefill_step(desc, q, q.stride(0), k, k.stride(0), v, v.stride(0), n, cu_seqlens_q, batch, max_seqlen_q,
                        context_lens, max_context_len, block_tables, max_pages_per_seq, q_norm_w, k_norm_w, eps,
                        rope_theta, scale, bufs.q_out, k_cache, v_cache, bufs.positions, bufs.slots, bufs.out,
                        bufs.workspace, stream=stream)
        return bufs.out
    _check_queries(desc, q, q_norm_w, k_norm_w)
    qa = _write_step(desc, bufs, q, k, v, cu_seqlens_q, context_lens, block_tables, k_cache, v_cache,
                     max_pages_per_seq, q_norm_w, k_norm_w, eps, rope_theta, stream)
    pa_decode(desc, qa, batch, k_cache, v_cache, block_tables, max_pages_per_seq, context_lens, max_context_len,
              scale, bufs.max_ctas, bufs.out, bufs.workspace, None, stream)
    return bufs.out


def _write_step(desc, bufs, q, k, v, cu_seqlens_q, context_lens, block_tables, k_cache, v_cache, max_pages_per_seq,
                q_norm_w, k_norm_w, eps, rope_theta, stream):
    """The step's K/V rows into the cache; returns the queries that attention takes."""
    n, batch = q.shape[0], context_lens.shape[0]
    if q_norm_w is not None:
        # slot mapping, norm, rotary and KV write in one kernel
        pa_prefill_qk_norm_rope_kv_write(desc, q, q.stride(0), k, k.stride(0), v, v.stride(0), n, cu_seqlens_q,
                                         batch, context_lens, block_tables, max_pages_per_seq, q_norm_w, k_norm_w,
                                         eps, rope_theta, bufs.q_out, k_cache, v_cache, bufs.positions, bufs.slots,
                                         stream)
        return bufs.q_out
    pa_slot_mapping(desc, batch, cu_seqlens_q, context_lens, block_tables, max_pages_per_seq, n, bufs.positions,
                    bufs.slots, stream)
    pa_kv_write(desc, k, k.stride(0), v, v.stride(0), n, bufs.slots, k_cache, v_cache, stream)
    return q


def _run_step_range(desc, kind, bufs, q, k, v, cu_seqlens_q, context_lens, block_tables, k_cache, v_cache, scale,
                    max_pages_per_seq, max_context_len, max_seqlen_q, q_norm_w, k_norm_w, eps, rope_theta, stream,
                    window, num_sinks, cu_groups, prefix_lens, max_prefix_len):
    """A step over a window, or with groups that share a prefix."""
    n, batch = q.shape[0], context_lens.shape[0]
    if window and cu_groups is not None:
        _refuse(PA_ERR_UNSUPPORTED, "a window and shared prefixes in one step")
    if bufs.group_size:
        _refuse(PA_ERR_UNSUPPORTED, "a 4-bit cache has no windowed and no shared-prefix attention")
    if cu_groups is not None and kind != "decode":
        _refuse(PA_ERR_UNSUPPORTED, "shared prefixes are a decode step's")
    if not 0 <= window < 2 ** 31 or (window and not 0 <= num_sinks < 2 ** 31):
        _refuse(PA_ERR_SHAPE, "a window is at least 1, the sinks at least 0, and both are below 2^31")
    if (kind != "decode" and n and torch_dtype(desc) is torch.bfloat16 and desc.head_dim == 128
            and desc.num_pages * desc.page_size >= 2 ** 31):
        _refuse(PA_ERR_UNSUPPORTED, "prefill in bf16 with head_dim 128 takes a cache of less than 2^31 rows")
    groups = 0
    if cu_groups is not None:
        groups = cu_groups.shape[0] - 1
        if prefix_lens is None:
            _refuse(PA_ERR_NULL, "groups without prefix lengths")
        if groups < 0 or prefix_lens.shape[0] < groups or not 0 <= max_prefix_len <= max_context_len:
            _refuse(PA_ERR_SHAPE, "cu_groups, prefix_lens or max_prefix_len out of range")
    _check_queries(desc, q, q_norm_w, k_norm_w)
    if q_norm_w is None:
        _check_rows(desc, bufs, n, k, v, k_cache, v_cache)

    def need():
        if not (n and batch):
            return 0
        if kind != "decode":
            return (pa_prefill_workspace_size(desc, batch, max_seqlen_q, n, max_context_len)
                    if bufs.workspace is not None else 0)
        nbytes = (pa_decode_window_workspace_size(desc, window, num_sinks, batch, max_context_len, bufs.max_ctas)
                  if window else pa_decode_shared_prefix_workspace_size(desc, groups, batch, max_prefix_len,
                                                                        max_context_len, bufs.max_ctas))
        if nbytes == 0:
            _refuse(PA_ERR_UNSUPPORTED, "decode does not take this descriptor, or there is no device")
        return nbytes

    _check_attention(desc, kind, bufs, q, batch, scale, max_pages_per_seq, max_context_len, max_seqlen_q,
                     q_norm_w is not None, need, positive_scale=cu_groups is not None)
    qa = _write_step(desc, bufs, q, k, v, cu_seqlens_q, context_lens, block_tables, k_cache, v_cache,
                     max_pages_per_seq, q_norm_w, k_norm_w, eps, rope_theta, stream)
    if kind != "decode":
        pa_prefill_varlen_window(desc, window, num_sinks, qa, cu_seqlens_q, batch, max_seqlen_q, n, k_cache, v_cache,
                                 block_tables, max_pages_per_seq, context_lens, max_context_len, scale, bufs.out,
                                 bufs.workspace, None, stream)
    elif window:
        pa_decode_window(desc, window, num_sinks, qa, batch, k_cache, v_cache, block_tables, max_pages_per_seq,
                         context_lens, max_context_len, scale, bufs.max_ctas, bufs.out, bufs.workspace, None, stream)
    else:
        pa_decode_shared_prefix(desc, groups, cu_groups, prefix_lens, max_prefix_len, qa, batch, k_cache, v_cache,
                                block_tables, max_pages_per_seq, context_lens, max_context_len, scale, bufs.max_ctas,
                                bufs.out, bufs.workspace, None, stream)
    return bufs.out


def _refuse(status: int, message: str):
    raise PagedAttnError("run_step", status, message)


def _check_queries(desc, q, q_norm_w, k_norm_w):
    """Both norm weights or neither; without them attention reads q itself, so its rows have to be packed."""
    if (q_norm_w is None) != (k_norm_w is None):
        _refuse(PA_ERR_NULL, "one norm weight without the other")
    n = q.shape[0]
    if q_norm_w is None and n and not (q[0].is_contiguous() and
                                       (n == 1 or q.stride(0) == desc.num_q_heads * desc.head_dim)):
        _refuse(PA_ERR_SHAPE, "without norm weights attention reads q itself, so its rows must be packed")


def _check_rows(desc, bufs, n, k, v, k_cache, v_cache):
    """What the write of a step's rows as they are (no norm weights) refuses, once their slots are enqueued."""
    if not n:
        return
    if not all(map(_at, (k, v, k_cache, v_cache))):
        _refuse(PA_ERR_NULL, "k, v or a cache is missing")
    if min(k.stride(0), v.stride(0)) < desc.num_kv_heads * desc.head_dim:
        _refuse(PA_ERR_SHAPE, "the rows of k or v overlap")
    size = torch_dtype(desc).itemsize
    if any(t.stride(0) * size % 16 for t in (k, v)) or any(_at(t) % 16 for t in (k, v, k_cache, v_cache)):
        _refuse(PA_ERR_ALIGN, "k, v, the stride of their rows or a cache is not 16-byte aligned")
    if bufs.group_size:
        _q4_cache_shapes("run_step", desc, bufs.group_size, k_cache, v_cache)
        for t in (k_cache, v_cache):
            if isinstance(t, torch.Tensor) and t.device != bufs.slots.device:
                _refuse(PA_ERR_UNSUPPORTED, f"a cache on {t.device}, buffers on {bufs.slots.device}")


def _check_step_q4(desc, kind, bufs, q, k, v, k_cache, v_cache, batch, scale, max_pages_per_seq, max_context_len,
                   max_seqlen_q, q_norm_w, k_norm_w):
    """What the attention of a step over a 4-bit cache would refuse once the step's rows are written: refused before
    anything is enqueued (with norm weights the write's own checks come first in its call)."""
    n = q.shape[0]
    _check_queries(desc, q, q_norm_w, k_norm_w)
    if q_norm_w is None:
        _check_rows(desc, bufs, n, k, v, k_cache, v_cache)

    def need():
        if kind == "decode":
            return (pa_decode_q4_workspace_size(desc, bufs.group_size, batch, max_context_len, bufs.max_ctas)
                    if batch else 0)
        st = bufs.staging
        if st is None:
            raise ValueError("the buffers were not allocated for a prefill step over a 4-bit cache")
        if batch > st.block_tables.shape[0] or max_context_len > st.max_pages * desc.page_size:
            raise ValueError("the step's batch or max_context_len is beyond what the buffers were allocated for")
        return (pa_prefill_workspace_size(st.desc, batch, max_seqlen_q, n, max_context_len)
                if n and bufs.workspace is not None else 0)

    _check_attention(desc, kind, bufs, q, batch, scale, max_pages_per_seq, max_context_len, max_seqlen_q,
                     q_norm_w is not None, need)


def _check_attention(desc, kind, bufs, q, batch, scale, max_pages_per_seq, max_context_len, max_seqlen_q, norm, need,
                     positive_scale=False):
    """What attention refuses once the step's rows are written: bounds, scale, alignment, and a workspace of less than
    ``need()`` bytes."""
    n = q.shape[0]
    if n and not 1 <= max_context_len <= max_pages_per_seq * desc.page_size:
        _refuse(PA_ERR_SHAPE, "max_context_len is not within 1 .. max_pages_per_seq * page_size")
    if not math.isfinite(scale) or ((kind != "decode" or positive_scale) and not scale > 0):
        _refuse(PA_ERR_SHAPE, "the scale is not finite, or not positive where prefill or a shared prefix needs it")
    if any(t is not None and t.data_ptr() % 16 for t in (bufs.out, bufs.q_out if norm else q)):
        _refuse(PA_ERR_ALIGN, "q or out is not 16-byte aligned")
    ws, need = bufs.workspace, need()
    if kind == "decode":
        if need and ws is None:
            _refuse(PA_ERR_WORKSPACE, "the buffers have no decode workspace")
    elif n and not (batch and 1 <= max_seqlen_q <= max_context_len):
        _refuse(PA_ERR_SHAPE, "tokens without requests, or max_seqlen_q is not within 1 .. max_context_len")
    if need and ws.numel() * ws.element_size() < need:
        _refuse(PA_ERR_WORKSPACE, "the buffers' workspace is smaller than this step needs")
    if ws is not None and ws.data_ptr() % 256:
        _refuse(PA_ERR_ALIGN, "the workspace is not 256-byte aligned")


def _run_step_q4(desc, kind, bufs, q, k, v, cu_seqlens_q, context_lens, block_tables, k_cache, v_cache, scale,
                 max_pages_per_seq, max_context_len, max_seqlen_q, q_norm_w, k_norm_w, eps, rope_theta, stream):
    """The step over a 4-bit cache.  What is skipped and flagged (``pa_read_device_errors``) is as over other caches: the
    staging cache's block tables have no page where the 4-bit cache's name none of it."""
    n, batch, gs = q.shape[0], context_lens.shape[0], bufs.group_size
    _check_step_q4(desc, kind, bufs, q, k, v, k_cache, v_cache, batch, scale, max_pages_per_seq, max_context_len,
                   max_seqlen_q, q_norm_w, k_norm_w)
    if q_norm_w is not None:
        pa_prefill_qk_norm_rope_kv_write_q4(desc, gs, q, q.stride(0), k, k.stride(0), v, v.stride(0), n,
                                            cu_seqlens_q, batch, context_lens, block_tables, max_pages_per_seq,
                                            q_norm_w, k_norm_w, eps, rope_theta, bufs.q_out, k_cache, v_cache,
                                            bufs.positions, bufs.slots, stream)
        q = bufs.q_out
    else:
        pa_slot_mapping(desc, batch, cu_seqlens_q, context_lens, block_tables, max_pages_per_seq, n, bufs.positions,
                        bufs.slots, stream)
        pa_kv_write_q4(desc, gs, k, k.stride(0), v, v.stride(0), n, bufs.slots, k_cache, v_cache, stream)
    if kind == "decode":
        pa_decode_q4(desc, gs, q, batch, k_cache, v_cache, block_tables, max_pages_per_seq, context_lens,
                     max_context_len, scale, bufs.max_ctas, bufs.out, bufs.workspace, None, stream)
        return bufs.out
    st = bufs.staging
    row = desc.num_kv_heads * desc.head_dim
    pa_kv_read_q4(desc, gs, batch, st.cu_rows, None, context_lens, block_tables, max_pages_per_seq,
                  batch * st.max_pages * desc.page_size, k_cache, v_cache, st.k, row, st.v, row, stream)
    pa_kv_read_q4_tables(desc, batch, st.cu_rows, block_tables, max_pages_per_seq, st.block_tables, st.max_pages, stream)
    pa_prefill_varlen(st.desc, q, cu_seqlens_q, batch, max_seqlen_q, n, st.k, st.v, st.block_tables, st.max_pages,
                      context_lens, max_context_len, scale, bufs.out, bufs.workspace, None, stream)
    return bufs.out
