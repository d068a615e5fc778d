// Decode attention with a range of each request's keys left out (a sliding
// window with sinks; a prefix that the requests of a group share), and decode
// for such groups.  The kernel is decode_kernel.cuh's: the chunks wholly
// inside the range are not in a request's chunk list, so neither their pages
// nor the table entries that name them are read; the rows of the range in the
// chunks at its two ends are not copied (tensor-core consumers) and have
// probability 0.  Bytes per request: min(L, sinks + window) K and V rows; HBM
// bound like the kernel over all keys.  256 requests of 128 to 8192 tokens over a
// window of 1024 (16 / 8 heads of 128): 155 us for 1.02 GB, 0.97 of a copy's rate; 64
// of 8192 to 32768 over 4096 (32 / 8): 158 us for 1.09 GB; DRAM reads equal the bytes
// that the windows hold.
#include <cmath>

#include "decode_kernel.cuh"
#include "prefix_plan.cuh"

namespace pa {

cudaError_t plan_decode_window(const pa_cache_desc& d, int batch, int max_ctx, int window, int sinks, int max_ctas,
                               DecodePlan* out) {
  const int64_t keys = static_cast<int64_t>(window) + sinks;
  if (keys >= max_ctx) return plan_decode(d, batch, max_ctx, max_ctas, out);  // nothing is left out
  // the sinks' last chunk and the window's first may both be partly filled
  cudaError_t e = plan_decode_keys<true>(d, batch, max_ctx, static_cast<int>(keys), 2, max_ctas, out);
  if (e != cudaSuccess) return e;
  // A CTA for each request saves the merge and the sums over the batch.  It pays
  // where a request has few keys, or where the requests about fill the CTAs that
  // fit (GPU us, shares of keys -> a CTA a request; 16 / 8 heads of 128, bf16):
  //   16 keys  1 request 6.6 -> 5.1   8: 7.6 -> 6.0   128: 10.6 -> 6.6   600: 22.5 -> 22.7
  //   64               7.8 -> 8.9       8.0 -> 9.7        14.5 -> 10.5        38.1 -> 38.2 (32: 10.3 -> 10.2)
  //   256              7.9 -> 23.9      9.0 -> 24.8       27.9 -> 25.7       104.7 -> 103.8
  // and fp32 (16 / 4 heads), slower by the key: 16 keys 6.8 -> 6.2, 64 keys 7.0 -> 14.0, 128 x 64 15.0 -> 15.5.
  // With 64 dims two CTAs fit an SM (16 / 8 heads, bf16; 16 / 4, fp32):
  //   bf16  16 keys  1 request 6.0 -> 4.4   128: 9.6 -> 5.7   600: 19.0 -> 13.4
  //         64               7.1 -> 7.1       12.3 -> 8.9       27.9 -> 23.5
  //         256              7.3 -> 16.8      20.6 -> 19.0      300: 34.3 -> 29.1
  //   fp32  16 keys          7.1 -> 5.0        9.5 -> 6.1       18.2 -> 7.8
  //         64               6.9 -> 9.1       12.0 -> 10.5      27.7 -> 18.0
  //         256              7.3 -> 25.3      20.2 -> 27.0      300: 35.5 -> 30.8
  const int few = d.dtype == PA_F32 ? 16 : 32;
  out->per_request = (keys <= few || (keys <= 2 * few && batch >= 32) ||
                      (keys <= 256 && 3 * static_cast<int64_t>(batch) >= 2 * out->slots && batch <= out->slots)) &&
                     (max_ctas == 0 || batch <= max_ctas);
  return cudaSuccess;
}

cudaError_t launch_decode_window(const pa_cache_desc& d, const DecodePlan& pl, const DecodeArgs& a, cudaStream_t s) {
  if (static_cast<int64_t>(a.window) + a.sinks >= a.max_context_len) return launch_decode(d, pl, a, s);
  const Fns f = get_fns<true>(d.dtype, d.head_dim, d.num_q_heads / d.num_kv_heads);
  if (!f.main) return cudaErrorInvalidValue;
  KParams p = decode_params(d, pl, a, d.num_kv_heads * d.head_dim * elem_bytes(d.dtype));
  p.window = a.window;
  p.sinks = a.sinks;
  void* args[] = {&p};
  return launch_decode_kernels<true>(f.main, f.merge, pl, p, args, s);
}

// ---------------------------------------------------------------------------
// Groups of requests that share a prefix.  Three kernels: the prefixes', whose
// tiles every query of a group meets at once (tcgen05 for bf16 with head_dim
// 128, else tile_attention.cu); the requests' own keys', beside it as its CTAs
// leave the SMs; the merge of both kernels' parts.  96 requests (32 / 8 heads of
// 128) in three groups behind 3000 to 9000 keys with 40 to 700 of their own: 64 us,
// 29 of them the first kernel; 128 behind 32768 with 20 to 300: 97 us, 70 of them.
// ---------------------------------------------------------------------------
namespace {

// out = sum_k 2^(lse_k - M) o_k / sum_k 2^(lse_k - M) over the parts of a
// request: the CTAs that had tiles of its unit of the prefix, then the CTAs that
// had chunks of its own keys.  merge_w warps per (request, q-head), each with a
// run of the parts, as decode_merge_kernel.  Which parts there are follows from
// the sums that the CTAs 0 of both grids leave: with every warp working them out
// from the lengths, a batch of 128 requests spent 40 us here.
template <typename T, int HD>
__global__ void __launch_bounds__(kMergeThreads)
    shared_merge_kernel(const KParams p, const PrefixShape s, const int64_t* costs, const float* o_pre,
                        const float* lse_pre) {
  constexpr int EL = HD / 32;
  constexpr int NWARP = kMergeThreads / 32;
  __shared__ float red[NWARP][32][EL + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int W = p.merge_w, item = warp / W, sub = warp - item * W;
  const int64_t u = static_cast<int64_t>(blockIdx.x) * (NWARP / W) + item;
  bool active = u < static_cast<int64_t>(p.B) * p.Hq;  // (all W warps of an item alike)
  const int b = active ? static_cast<int>(u / p.Hq) : 0;
  const int hq = active ? static_cast<int>(u - static_cast<int64_t>(b) * p.Hq) : 0;
  const int G = p.Hq / p.Hkv, h = hq / G;
  const int g = group_of(s.cu, s.n_groups, b);
  PrefixGroup gr{};
  if (active && g >= 0) gr = prefix_group(s, g);
  {
    const int L = p.ctx[b];
    const int cap = static_cast<int>(min(static_cast<int64_t>(p.max_ctx), static_cast<int64_t>(p.maxp) << p.log2P));
    active = active && L >= 1 && L <= cap && hole_of(p, b, L).hi >= 0;  // its lengths are consistent
  }
  pdl_wait();  // the parts and sums of both grids are written
  const int NC = p.cs[p.B], cb0 = p.cs[b], cb1 = p.cs[b + 1];
  const int64_t total = costs[s.n_groups];
  // the prefix's parts: np CTAs from f0 on
  int f0 = 0, np = 0;
  if (gr.cost > 0) {
    const int ctas = static_cast<int>(costs[s.n_groups + 1]);
    const PrefixUnit unit = prefix_unit(s, gr, costs[g], h, (b - gr.s0) / s.TQ / 2);
    f0 = prefix_cta_of(unit.start, total, ctas);
    np = prefix_cta_of(unit.start + static_cast<int64_t>(gr.nt - 1) * unit.cost, total, ctas) - f0 + 1;
  }
  // the request's own: ns CTAs from c0 on
  int c0 = 0, ns = 0;
  if (cb1 > cb0) {
    const int n_ctas = sharing_ctas<true>(p, NC);
    c0 = static_cast<int>(((static_cast<int64_t>(cb0) + 1) * n_ctas + NC - 1) / NC) - 1;
    ns = static_cast<int>((static_cast<int64_t>(cb1) * n_ctas + NC - 1) / NC) - c0;
  }
  // without a prefix a single CTA's result is the output already
  active = active && (np > 0 || ns > 1);
  const int parts = np + ns;
  const int64_t pre_row = np > 0 ? prefix_part_row(s, gr.s0, gr.n, h, f0, p.Hq, G) + (b - gr.s0) * G + hq - h * G : 0;
  const int64_t own_row = static_cast<int64_t>(c0 + b) * p.Hq + hq;
  auto row_of = [&](int k) { return k < np ? pre_row + static_cast<int64_t>(k) * s.unit_rows
                                           : own_row + static_cast<int64_t>(k - np) * p.Hq; };
  auto lse_of = [&](int k) { return k < np ? lse_pre[row_of(k)] : p.lse_part[row_of(k)]; };
  float acc[EL];
#pragma unroll
  for (int e = 0; e < EL; ++e) acc[e] = 0.f;
  float wsum = 0.f;
  if (active) {
    const int per = (parts + W - 1) / W;
    const int k_begin = sub * per, k_end = min(parts, k_begin + per);
    float v[8][EL];
    auto load = [&](int k0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int k = k0 + i;
        if (k < k_end) {
          const float* src = (k < np ? o_pre : p.o_part) + row_of(k) * HD + lane * EL;
          if constexpr (EL == 4) {
            const float4 ov = *reinterpret_cast<const float4*>(src);
            v[i][0] = ov.x, v[i][1] = ov.y, v[i][2] = ov.z, v[i][3] = ov.w;
          } else {
            const float2 ov = *reinterpret_cast<const float2*>(src);
            v[i][0] = ov.x, v[i][1] = ov.y;
          }
        }
      }
    };
    load(k_begin);
    // the first 32 parts' log-sum-exps stay in the lanes
    const float lse_mine = lane < parts ? lse_of(lane) : -INFINITY;
    float M = fmaxf(lse_mine, -INFINITY);
    bool nan = lse_mine != lse_mine;
    for (int k = lane + 32; k < parts; k += 32) {
      const float x = lse_of(k);
      M = fmaxf(M, x);
      nan |= x != x;
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    M = merge_maximum(M, nan);
    if (M != -INFINITY) {
      const float w_first = exp2f(lse_mine - M);
      for (int k0 = k_begin; k0 < k_end; k0 += 8) {
        if (k0 != k_begin) load(k0);
        const int k = k0 + lane;
        float w_mine = 0.f;
        if (parts > 32 && lane < 8 && k < k_end) w_mine = exp2f(lse_of(k) - M);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float w = parts > 32 ? __shfl_sync(0xffffffffu, w_mine, i)
                                     : __shfl_sync(0xffffffffu, w_first, (k0 + i) & 31);
          if (k0 + i < k_end) {
#pragma unroll
            for (int e = 0; e < EL; ++e) acc[e] += w * v[i][e];
            wsum += w;
          }
        }
      }
    }
  }
  if (W > 1) {
#pragma unroll
    for (int e = 0; e < EL; ++e) red[warp][lane][e] = acc[e];
    red[warp][lane][EL] = wsum;
    cta_sync();
    if (sub != 0) return;
    for (int w2 = 1; w2 < W; ++w2) {
#pragma unroll
      for (int e = 0; e < EL; ++e) acc[e] += red[warp + w2][lane][e];
      wsum += red[warp + w2][lane][EL];
    }
  }
  if (!active) return;
  const float inv = wsum > 0.f ? 1.f / wsum : 0.f;
  const int64_t e0 = (static_cast<int64_t>(b) * p.Hq + hq) * HD + lane * EL;
#pragma unroll
  for (int e = 0; e < EL; e += 2) {
    if constexpr (sizeof(T) == 2)
      *reinterpret_cast<uint32_t*>(p.out + (e0 + e) * 2) = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
    else
      *reinterpret_cast<float2*>(p.out + (e0 + e) * 4) = make_float2(acc[e] * inv, acc[e + 1] * inv);
  }
}

bool prefix_on_tcgen05(const pa_cache_desc& d) { return d.dtype == PA_BF16 && d.head_dim == 128; }

}  // namespace

PrefixShape prefix_shape(const pa_cache_desc& d, const SharedArgs& a, const SharedPlan& pl) {
  PrefixShape s{};
  s.cu = a.cu_groups;
  s.pre = a.prefix_lens;
  s.ctx = a.context_lens;
  s.n_groups = a.n_groups;
  s.B = a.batch;
  s.max_prefix = a.max_prefix;
  s.cap_ctx = static_cast<int32_t>(
      std::min<int64_t>(a.max_context_len, static_cast<int64_t>(a.max_pages) * d.page_size));
  s.TQ = pl.TQ;
  s.Hkv = d.num_kv_heads;
  s.cost_pair = pl.cost_pair;
  s.cost_one = pl.cost_one;
  s.min_share = pl.min_share;
  s.unit_rows = pl.unit_rows;
  return s;
}

cudaError_t plan_shared(const pa_cache_desc& d, int n_groups, int batch, int max_prefix, int max_ctx, int max_ctas,
                        SharedPlan* out) {
  SharedPlan pl;
  const bool shared = n_groups > 0 && max_prefix > 0;
  cudaError_t e = shared ? plan_decode_keys<true>(d, batch, max_ctx, max_ctx, 0, max_ctas, &pl.suffix)
                         : plan_decode(d, batch, max_ctx, max_ctas, &pl.suffix);
  if (e != cudaSuccess) return e;
  pl.ws_bytes = align_up(pl.suffix.ws_bytes, 256);
  if (shared) {
    DeviceInfo di;
    if ((e = current_device_info(&di)) != cudaSuccess) return e;
    const int G = d.num_q_heads / d.num_kv_heads;
    const bool tc = prefix_on_tcgen05(d);
    pl.unit_rows = tc ? 256 : prefix_tile_rows(d);
    pl.TQ = pl.unit_rows / 2 / G;
    // a tile of one q-tile alone takes about 0.7 of the time that one of two takes
    pl.cost_pair = tc ? 10 : 1;
    pl.cost_one = tc ? 7 : 1;
    pl.min_share = tc ? 14 : 1;
    const int most = di.sm_count * (tc ? 1 : 2);
    pl.prefix_ctas = max_ctas > 0 ? std::min(max_ctas, most) : most;
    // Few keys in all (by the bounds): one decode over prefixes and own keys reads
    // a prefix once for each request, but spares a kernel and the larger merge.
    // Estimates, us, beyond what both cost; measured, us (each, once; q- / kv-heads
    // of dims, requests / groups, prefix):
    //   bf16 16/8 of 128   4/1  1024  12.8 19.0    16/1  1024  19.2 19.3    64/1   256  19.5 23.0
    //                     64/1  1024  44.9 25.2    24/3  4096  62.0 27.9   128/7   256  31.5 26.9
    //   bf16 16/8 of 64    4/1  1024  11.3 13.1    16/1  1024  14.9 14.0    24/3  4096  33.5 20.6
    //   fp32 16/4 of 128  16/1  1024  19.0 35.4    16/1  4096  39.3 41.2    16/1 16384 123.1 115.4
    // Of 55 more in 64 dims and fp32 (16/8, 32/8, 16/4; 4 to 128 requests in 1 to 7
    // groups behind 256 to 16384 tokens) the rule takes one that is slower by more
    // than 15% twice: bf16 16/8 of 64, 16/1 512 13.3 11.4; 32/8 of 64, 64/1 256 18.3 14.5.
    const double row = 2.0 * d.num_kv_heads * d.head_dim * elem_bytes(d.dtype);
    const double each_us = batch * static_cast<double>(max_prefix) * row / 6.0e6;
    const double units = std::ceil(static_cast<double>(batch) / n_groups * G / pl.unit_rows) * n_groups * d.num_kv_heads;
    const double tile_us = tc ? 2 : d.dtype == PA_BF16 ? 2.8 : d.head_dim == 64 ? 14 : 24;  // 128 keys of a unit
    const double once_us = (tc ? 7 + 0.09 * batch : 4) + std::ceil(units * ((max_prefix + 127) / 128) / most) * tile_us;
    pl.through_rep = each_us < once_us;
    // (the parts' room is in the size either way: a workspace for the largest bounds serves smaller ones)
    const int64_t rows = static_cast<int64_t>(batch) * d.num_q_heads + static_cast<int64_t>(pl.prefix_ctas) * pl.unit_rows;
    if (rows >= int64_t(1) << 31) return cudaErrorInvalidValue;
    // TMA coordinates are 32-bit: the cache rows must be addressable
    if (tc && d.num_pages * d.page_size >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
    pl.off_costs = pl.ws_bytes;
    pl.off_lse = align_up(pl.off_costs + (static_cast<size_t>(n_groups) + 2) * 8, 256);
    pl.off_o = align_up(pl.off_lse + static_cast<size_t>(rows) * 4, 256);
    pl.ws_bytes = align_up(pl.off_o + static_cast<size_t>(rows) * d.head_dim * 4, 256);
  }
  *out = pl;
  return cudaSuccess;
}

cudaError_t launch_shared(const pa_cache_desc& d, const SharedPlan& pl, const SharedArgs& a, cudaStream_t s) {
  DecodeArgs da{};
  da.q = a.q;
  da.k_cache = a.k_cache;
  da.v_cache = a.v_cache;
  da.block_tables = a.block_tables;
  da.context_lens = a.context_lens;
  da.out = a.out;
  da.workspace = a.workspace;
  da.err = a.err;
  da.batch = a.batch;
  da.max_pages = a.max_pages;
  da.max_context_len = a.max_context_len;
  da.scale = a.scale;
  da.keep_nan = true;
  if (pl.prefix_ctas == 0) return launch_decode(d, pl.suffix, da, s);
  const Fns f = get_fns<true>(d.dtype, d.head_dim, d.num_q_heads / d.num_kv_heads);
  if (!f.main) return cudaErrorInvalidValue;
  KParams p = decode_params(d, pl.suffix, da, d.num_kv_heads * d.head_dim * elem_bytes(d.dtype));
  void* args[] = {&p};
  p.cu_groups = a.cu_groups;
  p.prefix_lens = a.prefix_lens;
  p.n_groups = a.n_groups;
  p.max_prefix = a.max_prefix;
  if (pl.through_rep) {
    p.through_rep = 1;
    return launch_decode_kernels<true>(f.main, f.merge, pl.suffix, p, args, s);
  }
  cudaError_t e = prefix_on_tcgen05(d) ? launch_prefix_tc(d, a, pl, s) : launch_prefix_tile(d, a, pl, s);
  if (e != cudaSuccess) return e;
  const int threads = (pl.suffix.nw + 1) * 32;
  if (!p.inline_plan) {
    decode_plan_kernel<true><<<1, kPlanThreads, 0, s>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  // The decode grid reads nothing that the kernel before it writes (but for the
  // plan kernel's sums, which it waits for), and waits for it before it ends.
  e = launch_after_previous(f.main, dim3(pl.suffix.n_ctas), dim3(threads), pl.suffix.smem_bytes, s, args);
  if (e != cudaSuccess) return e;
  // warps per (request, q-head): about one per 8 parts (the CTAs of a kv-head's
  // one group, and of a request when all are equally long), where there are few
  const int parts = pl.prefix_ctas / d.num_kv_heads + pl.suffix.n_ctas / std::max(1, p.B);
  const bool few = static_cast<int64_t>(p.B) * p.Hq < 2048;
  p.merge_w = few && parts >= 24 ? 4 : few && parts >= 12 ? 2 : 1;
  PrefixShape shape = prefix_shape(d, a, pl);
  char* ws = static_cast<char*>(a.workspace);
  const int64_t* costs = reinterpret_cast<const int64_t*>(ws + pl.off_costs);
  const float* o_pre = reinterpret_cast<const float*>(ws + pl.off_o);
  const float* lse_pre = reinterpret_cast<const float*>(ws + pl.off_lse);
  void* margs[] = {&p, &shape, &costs, &o_pre, &lse_pre};
  const int64_t items = static_cast<int64_t>(p.B) * p.Hq;
  const int per_cta = kMergeThreads / 32 / p.merge_w;
  const void* merge =
      d.dtype == PA_BF16 ? (d.head_dim == 128 ? reinterpret_cast<const void*>(shared_merge_kernel<__nv_bfloat16, 128>)
                                              : reinterpret_cast<const void*>(shared_merge_kernel<__nv_bfloat16, 64>))
                         : (d.head_dim == 128 ? reinterpret_cast<const void*>(shared_merge_kernel<float, 128>)
                                              : reinterpret_cast<const void*>(shared_merge_kernel<float, 64>));
  return launch_after_previous(merge, dim3(static_cast<unsigned>((items + per_cta - 1) / per_cta)),
                               dim3(kMergeThreads), 0, s, margs);
}

}  // namespace pa
