// Batched GQA decode attention over all of each request's keys: the kernel of
// decode_kernel.cuh without a range left out.
#include "decode_kernel.cuh"

namespace pa {

cudaError_t plan_decode(const pa_cache_desc& d, int batch, int max_ctx, int max_ctas, DecodePlan* out) {
  return plan_decode_keys<false>(d, batch, max_ctx, max_ctx, 0, max_ctas, out);
}

cudaError_t launch_decode(const pa_cache_desc& d, const DecodePlan& pl, const DecodeArgs& a, cudaStream_t s) {
  const int G = d.num_q_heads / d.num_kv_heads;
  const Fns f = get_fns<false>(d.dtype, d.head_dim, G);
  if (!f.main) return cudaErrorInvalidValue;
  KParams p = decode_params(d, pl, a, d.num_kv_heads * d.head_dim * elem_bytes(d.dtype));
  void* args[] = {&p};
  return launch_decode_kernels<false>(f.main, f.merge, pl, p, args, s);
}

}  // namespace pa
