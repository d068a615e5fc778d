// The entry points of attention over part of each request's keys, or over keys
// that requests share: argument checks and dispatch.
#include <cuda_runtime.h>
#include <math.h>

#include "pa_internal.h"

namespace pa {
namespace {

pa_status check_window(int32_t window, int32_t num_sinks) {
  return window < 1 || num_sinks < 0 ? PA_ERR_SHAPE : PA_OK;
}

// The bound on the contexts that the kernels take: they round lengths up to tiles of
// up to 128 keys in 32 bits.  (Longer contexts are skipped and flagged.)
int32_t most_keys(int32_t max_context_len) { return max_context_len < 0x7fffff80 ? max_context_len : 0x7fffff80; }

pa_status check_workspace(const void* workspace) {
  if (!workspace) return PA_ERR_WORKSPACE;
  return (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ? PA_ERR_ALIGN : PA_OK;
}

// Plan, parameters and launch of a windowed decode whose arguments are checked.
pa_status decode_window(const pa_cache_desc* desc, DecodeArgs& a, int32_t max_ctas, size_t workspace_bytes,
                        pa_stream_t stream) {
  pa_status st = check_workspace(a.workspace);
  if (st != PA_OK) return st;
  DecodePlan pl;
  cudaError_t e = plan_decode_window(*desc, a.batch, a.max_context_len, a.window, a.sinks, max_ctas, &pl);
  if (e == cudaErrorInvalidValue) return PA_ERR_UNSUPPORTED;
  if (e != cudaSuccess) return cuda_fail(e);
  if (workspace_bytes < pl.ws_bytes) return PA_ERR_WORKSPACE;
  if ((st = prepare(&a.err)) != PA_OK) return st;
  e = launch_decode_window(*desc, pl, a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PA_OK : cuda_fail(e);
}

DecodeArgs decode_args(const void* q, int32_t batch, const void* k_cache, const void* v_cache,
                       const int32_t* block_tables, int32_t max_pages_per_seq, const int32_t* context_lens,
                       int32_t max_context_len, float scale, void* out, void* workspace) {
  DecodeArgs a{};
  a.q = q;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.out = out;
  a.workspace = workspace;
  a.batch = batch;
  a.max_pages = max_pages_per_seq;
  a.max_context_len = most_keys(max_context_len);
  a.scale = scale;
  a.keep_nan = true;  // whatever the bounds leave out
  return a;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" {

size_t pa_decode_window_workspace_size(const pa_cache_desc* desc, int32_t window, int32_t num_sinks, int32_t batch,
                                       int32_t max_context_len, int32_t max_ctas) {
  if (check_desc(desc) != PA_OK || check_window(window, num_sinks) != PA_OK) return 0;
  if (batch < 1 || max_context_len < 1 || max_ctas < 0) return 0;
  DecodePlan pl;
  if (plan_decode_window(*desc, batch, most_keys(max_context_len), window, num_sinks, max_ctas, &pl) != cudaSuccess)
    return 0;
  return pl.ws_bytes;
}

pa_status pa_decode_window(const pa_cache_desc* desc, int32_t window, int32_t num_sinks, const void* q, int32_t batch,
                           const void* k_cache, const void* v_cache, const int32_t* block_tables,
                           int32_t max_pages_per_seq, const int32_t* context_lens, int32_t max_context_len,
                           float scale, int32_t max_ctas, void* out, void* workspace, size_t workspace_bytes,
                           pa_stream_t stream) {
  pa_status st = check_decode_args(desc, q, batch, k_cache, v_cache, block_tables, max_pages_per_seq, context_lens,
                                   max_context_len, scale, max_ctas, out);
  if (st != PA_OK) return st;
  if ((st = check_window(window, num_sinks)) != PA_OK || batch == 0) return st;
  DecodeArgs a = decode_args(q, batch, k_cache, v_cache, block_tables, max_pages_per_seq, context_lens,
                             max_context_len, scale, out, workspace);
  a.window = window;
  a.sinks = num_sinks;
  return decode_window(desc, a, max_ctas, workspace_bytes, stream);
}

pa_status pa_decode_kv_write_window(const pa_cache_desc* desc, int32_t window, int32_t num_sinks, const void* q,
                                    const void* k_new, int64_t k_row_stride, const void* v_new, int64_t v_row_stride,
                                    int32_t batch, void* k_cache, void* v_cache, const int32_t* block_tables,
                                    int32_t max_pages_per_seq, const int32_t* context_lens, int32_t max_context_len,
                                    float scale, int32_t max_ctas, int64_t* slot_mapping, void* out, void* workspace,
                                    size_t workspace_bytes, pa_stream_t stream) {
  pa_status st = check_decode_args(desc, q, batch, k_cache, v_cache, block_tables, max_pages_per_seq, context_lens,
                                   max_context_len, scale, max_ctas, out);
  if (st != PA_OK) return st;
  if ((st = check_window(window, num_sinks)) != PA_OK || batch == 0) return st;
  if (!k_new || !v_new) return PA_ERR_NULL;
  const int64_t re = row_elems(desc);
  if (k_row_stride < re || v_row_stride < re) return PA_ERR_SHAPE;
  if (!stride_ok(desc, k_row_stride, re) || !stride_ok(desc, v_row_stride, re)) return PA_ERR_ALIGN;
  if (!aligned16(k_new) || !aligned16(v_new)) return PA_ERR_ALIGN;
  if (desc->num_pages * desc->page_size >= (int64_t(1) << 31)) return PA_ERR_UNSUPPORTED;
  DecodeArgs a = decode_args(q, batch, k_cache, v_cache, block_tables, max_pages_per_seq, context_lens,
                             max_context_len, scale, out, workspace);
  a.window = window;
  a.sinks = num_sinks;
  a.k_new = k_new;
  a.v_new = v_new;
  a.k_new_stride_bytes = k_row_stride * elem_bytes(desc->dtype);
  a.v_new_stride_bytes = v_row_stride * elem_bytes(desc->dtype);
  a.slot_out = slot_mapping;
  return decode_window(desc, a, max_ctas, workspace_bytes, stream);
}

pa_status pa_prefill_varlen_window(const pa_cache_desc* desc, int32_t window, int32_t num_sinks, const void* q,
                                   const int32_t* cu_seqlens_q, int32_t batch, int32_t max_seqlen_q,
                                   int64_t num_tokens, const void* k_cache, const void* v_cache,
                                   const int32_t* block_tables, int32_t max_pages_per_seq,
                                   const int32_t* context_lens, int32_t max_context_len, float scale, void* out,
                                   void* workspace, size_t workspace_bytes, pa_stream_t stream) {
  pa_status st = check_desc(desc);
  if (st != PA_OK) return st;
  if ((st = check_window(window, num_sinks)) != PA_OK) return st;
  PrefillArgs a;
  st = prefill_args(desc, q, cu_seqlens_q, batch, max_seqlen_q, num_tokens, k_cache, v_cache, block_tables,
                    max_pages_per_seq, context_lens, max_context_len, scale, out, workspace, workspace_bytes, &a);
  if (st != PA_OK || a.num_tokens == 0) return st;
  a.max_context_len = most_keys(max_context_len);
  a.window = window;
  a.sinks = num_sinks;
  if ((st = prepare(&a.err)) != PA_OK) return st;
  cudaError_t e = launch_prefill(*desc, a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PA_OK : cuda_fail(e);
}

size_t pa_decode_shared_prefix_workspace_size(const pa_cache_desc* desc, int32_t num_groups, int32_t batch,
                                              int32_t max_prefix_len, int32_t max_context_len, int32_t max_ctas) {
  if (check_desc(desc) != PA_OK || num_groups < 0 || batch < 1 || max_prefix_len < 0 || max_context_len < 1 ||
      max_ctas < 0)
    return 0;
  SharedPlan pl;
  if (plan_shared(*desc, num_groups, batch, max_prefix_len, max_context_len, max_ctas, &pl) != cudaSuccess) return 0;
  return pl.ws_bytes;
}

pa_status pa_decode_shared_prefix(const pa_cache_desc* desc, int32_t num_groups, const int32_t* cu_groups,
                                  const int32_t* prefix_lens, int32_t max_prefix_len, const void* q, int32_t batch,
                                  const void* k_cache, const void* v_cache, const int32_t* block_tables,
                                  int32_t max_pages_per_seq, const int32_t* context_lens, int32_t max_context_len,
                                  float scale, int32_t max_ctas, void* out, void* workspace, size_t workspace_bytes,
                                  pa_stream_t stream) {
  pa_status st = check_decode_args(desc, q, batch, k_cache, v_cache, block_tables, max_pages_per_seq, context_lens,
                                   max_context_len, scale, max_ctas, out);
  if (st != PA_OK) return st;
  if (num_groups < 0 || max_prefix_len < 0) return PA_ERR_SHAPE;
  if (batch == 0) return PA_OK;
  if (max_prefix_len > max_context_len) return PA_ERR_SHAPE;
  if (!(scale > 0.f)) return PA_ERR_SHAPE;  // the tensor-core kernel takes the maximum before it scales
  if (num_groups > 0 && (!cu_groups || !prefix_lens)) return PA_ERR_NULL;
  if ((st = check_workspace(workspace)) != PA_OK) return st;
  SharedPlan pl;
  cudaError_t e = plan_shared(*desc, num_groups, batch, max_prefix_len, max_context_len, max_ctas, &pl);
  if (e == cudaErrorInvalidValue) return PA_ERR_UNSUPPORTED;
  if (e != cudaSuccess) return cuda_fail(e);
  if (workspace_bytes < pl.ws_bytes) return PA_ERR_WORKSPACE;
  SharedArgs a{};
  a.q = q;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.cu_groups = cu_groups;
  a.prefix_lens = prefix_lens;
  a.out = out;
  a.workspace = workspace;
  a.n_groups = num_groups;
  a.max_prefix = max_prefix_len;
  a.batch = batch;
  a.max_pages = max_pages_per_seq;
  a.max_context_len = most_keys(max_context_len);
  a.scale = scale;
  if ((st = prepare(&a.err)) != PA_OK) return st;
  e = launch_shared(*desc, pl, a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PA_OK : cuda_fail(e);
}

}  // extern "C"
