// Decode attention with a range of each request's keys left out: a sliding
// window with sinks.  The kernel is decode_kernel.cuh's: the chunks wholly
// inside the range are not in a request's chunk list, so neither their pages
// nor the table entries that name them are read; the rows of the range in the
// chunks at its two ends are not copied (tensor-core consumers) and have
// probability 0.  Bytes per request: min(L, sinks + window) K and V rows; HBM
// bound like the kernel over all keys.
#include "decode_kernel.cuh"

namespace pa {

cudaError_t plan_decode_window(const pa_cache_desc& d, int batch, int max_ctx, int window, int sinks, int max_ctas,
                               DecodePlan* out) {
  // the sinks' last chunk and the window's first may both be partly filled
  const int64_t keys = static_cast<int64_t>(window) + sinks;
  const bool all = keys >= max_ctx;
  return plan_decode_keys<true>(d, batch, all ? max_ctx : static_cast<int>(keys), all ? 0 : 2, max_ctas, out);
}

cudaError_t launch_decode_window(const pa_cache_desc& d, const DecodePlan& pl, const DecodeArgs& a, cudaStream_t s) {
  const Fns f = get_fns<true>(d.dtype, d.head_dim, d.num_q_heads / d.num_kv_heads);
  if (!f.main) return cudaErrorInvalidValue;
  KParams p = decode_params(d, pl, a, d.num_kv_heads * d.head_dim * elem_bytes(d.dtype));
  p.window = a.window;
  p.sinks = a.sinks;
  void* args[] = {&p};
  return launch_decode_kernels<true>(f.main, f.merge, pl, p, args, s);
}

}  // namespace pa
