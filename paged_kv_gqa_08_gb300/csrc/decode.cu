// Batched GQA decode attention over all of each request's keys: the kernel of
// decode_kernel.cuh without a range left out.
#include "decode_kernel.cuh"

namespace pa {

cudaError_t plan_decode(const pa_cache_desc& d, int batch, int max_ctx, int max_ctas, DecodePlan* out) {
  return plan_decode_keys<false>(d, batch, max_ctx, max_ctx, 0, max_ctas, out);
}

namespace {

template <typename T, int HD>
const void* merge_with_nan() {
  return reinterpret_cast<const void*>(decode_merge_kernel<T, HD, false, true>);
}

}  // namespace

cudaError_t launch_decode(const pa_cache_desc& d, const DecodePlan& pl, const DecodeArgs& a, cudaStream_t s) {
  const int G = d.num_q_heads / d.num_kv_heads;
  Fns f = get_fns<false>(d.dtype, d.head_dim, G);
  if (!f.main) return cudaErrorInvalidValue;
  if (a.keep_nan)
    f.merge = d.dtype == PA_BF16 ? (d.head_dim == 128 ? merge_with_nan<__nv_bfloat16, 128>() : merge_with_nan<__nv_bfloat16, 64>())
                                 : (d.head_dim == 128 ? merge_with_nan<float, 128>() : merge_with_nan<float, 64>());
  KParams p = decode_params(d, pl, a, d.num_kv_heads * d.head_dim * elem_bytes(d.dtype));
  void* args[] = {&p};
  return launch_decode_kernels<false>(f.main, f.merge, pl, p, args, s);
}

}  // namespace pa
