// What the decode kernels share, whatever the cache holds (bf16 / fp32 rows in
// decode.cu, 4-bit rows in decode_q4.cu): the kernels' parameters, the plan
// (chunk prefix sums, each CTA's share), the log-sum-exp merge of the shares'
// partial results, and the host side of a launch.
#pragma once

#include <math.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

#include "pa_common.cuh"

namespace pa {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kInlinePlanMax = 512;  // batches the decode CTAs plan themselves (else a plan kernel runs first)
constexpr int kMergeThreads = 128;

struct KParams {
  const char* q;
  const char* k_cache;
  const char* v_cache;
  const int32_t* bt;
  const int32_t* ctx;
  char* out;
  float* o_part;
  float* lse_part;
  int32_t* cs;       // [B+1] chunk prefix sums
  int32_t* cta_seq;  // [n_ctas] first request of each CTA
  unsigned int* err;
  int64_t num_pages;
  int32_t B, Hq, Hkv, P, maxp, max_ctx, n_ctas;
  int32_t log2P, log2T;
  int32_t row_bytes;    // Hkv * HD * E, one token of the cache
  int32_t row_pitch;    // shared-memory bytes per token row of a stage (row_bytes, + 16 for the MMA consumers)
  int32_t chunk_bytes;  // T * row_pitch
  uint32_t off_bar, off_meta, off_p, off_alpha, off_ml, off_abort;
  uint32_t off_cs;      // [kInlinePlanMax + 1] chunk prefix sums, then [32] warp totals (inline plan)
  int32_t inline_plan;  // 1: no plan kernel ran; every CTA computes the prefix sums itself
  int32_t p_row;        // floats per token row of the probability tile
  float scale_log2;     // softmax scale * log2(e)
  int32_t merge_w;      // warps per (request, q-head) in the merge kernel: 1, 2 or 4
  // Fused KV write (k_new != nullptr): the new token of request b is row b of
  // k_new / v_new; it is attended from there and stored into its cache slot
  // (position context_lens[b] - 1) by the CTA that owns the request's last chunk.
  const char* k_new;
  const char* v_new;
  int64_t k_new_stride, v_new_stride;  // bytes
  int64_t* slot_out;                   // optional: the slot written for request b
};

// First request whose chunks extend past chunk x0 (cs: the prefix sums).
__device__ __forceinline__ int first_request(const int32_t* cs, int B, int64_t x0) {
  int lo = 0, hi = B;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (cs[mid + 1] > x0) hi = mid; else lo = mid + 1;
  }
  return lo;
}

// ---------------------------------------------------------------------------
// plan: chunk prefix sums and each CTA's first request
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kPlanThreads) decode_plan_kernel(const KParams p) {
  __shared__ int32_t warp_tot[kPlanThreads / 32];
  __shared__ int32_t carry;
  pdl_trigger();  // the decode kernel may start launching; it waits for this plan
  const int tid = threadIdx.x;
  const int T = 1 << p.log2T;
  const int cap = static_cast<int>(min(static_cast<int64_t>(p.max_ctx), static_cast<int64_t>(p.maxp) << p.log2P));
  if (tid == 0) carry = 0;
  cta_sync();
  for (int base = 0; base < p.B; base += kPlanThreads) {
    const int b = base + tid;
    int cnt = 0;
    if (b < p.B) {
      const int L = p.ctx[b];
      if (L >= 1 && L <= cap) {
        cnt = (L + T - 1) >> p.log2T;
      } else {
        // length 0 is a padding row: nothing is read, stored or written for it
        if (L != 0) raise_flag(p.err, PA_DEVERR_BAD_LENGTH);
        if (p.k_new != nullptr && p.slot_out) p.slot_out[b] = -1;
      }
    }
    int x = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if ((tid & 31) >= o) x += y;
    }
    if ((tid & 31) == 31) warp_tot[tid >> 5] = x;
    cta_sync();
    if (tid < 32) {
      int w = warp_tot[tid];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, w, o);
        if (tid >= o) w += y;
      }
      warp_tot[tid] = w;
    }
    cta_sync();
    const int incl = x + ((tid >> 5) ? warp_tot[(tid >> 5) - 1] : 0) + carry;
    if (b < p.B) p.cs[b + 1] = incl;
    cta_sync();
    if (tid == kPlanThreads - 1) carry = incl;
    cta_sync();
  }
  if (tid == 0) p.cs[0] = 0;
  cta_sync();
  const int NC = carry;
  for (int c = tid; c < p.n_ctas; c += kPlanThreads)
    p.cta_seq[c] = first_request(p.cs, p.B, (static_cast<int64_t>(c) * NC) / p.n_ctas);
}

// The plan kernel's prefix sums, computed by every thread of a decode CTA into
// its shared memory (B <= kInlinePlanMax): each thread sums the chunk counts
// of a run of consecutive requests, the runs' totals are scanned across the
// CTA, then each thread writes its run's prefix sums.  CTA 0 also does the
// plan kernel's side work: it flags bad lengths and marks the slots of rows it
// skips.  (The merge kernel works the sums out for itself.)
__device__ __forceinline__ void plan_in_cta(const KParams& p, int32_t* cs_s, int32_t* warp_tot, bool first) {
  const int nthr = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int T = 1 << p.log2T;
  const int cap = static_cast<int>(min(static_cast<int64_t>(p.max_ctx), static_cast<int64_t>(p.maxp) << p.log2P));
  const int per = (p.B + nthr - 1) / nthr;
  const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
  int sum = 0;
  for (int b = b0; b < b1; ++b) {
    const int L = p.ctx[b];
    int cnt = 0;
    if (L >= 1 && L <= cap) {
      cnt = (L + T - 1) >> p.log2T;
    } else if (first) {
      // length 0 is a padding row: nothing is read, stored or written for it
      if (L != 0) raise_flag(p.err, PA_DEVERR_BAD_LENGTH);
      if (p.k_new != nullptr && p.slot_out) p.slot_out[b] = -1;
    }
    cs_s[b + 1] = cnt;
    sum += cnt;
  }
  int x = sum;  // inclusive scan of the runs' totals: within the warp, then over the warps
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_tot[warp] = x;
  cta_sync();
  if (warp == 0) {
    int w = lane < (nthr >> 5) ? warp_tot[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    warp_tot[lane] = w;
  }
  cta_sync();
  int run = x - sum + (warp ? warp_tot[warp - 1] : 0);
  for (int b = b0; b < b1; ++b) {
    run += cs_s[b + 1];
    cs_s[b + 1] = run;
  }
  if (tid == 0) cs_s[0] = 0;
  cta_sync();
}

// Time-only bounded wait used when draining copies after an abort.
PA_DEVINL void drain_wait(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (global_timer_ns() - t0 > kWaitLimitNs) return;
  }
}

// 2^x on the special-function unit (PTX ex2.approx, results below 2^-126 as 0; x is
// at most 0 in decode.cu and the merges, at most 11 in decode_q4.cu).  exp2f gives the
// same bits wherever the result is no subnormal.
PA_DEVINL float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ---------------------------------------------------------------------------
// log-sum-exp merge of the partials of requests cut across CTAs.  merge_w
// warps per (request, q-head): each takes a contiguous range of the partials,
// a lane owns HD/32 elements of the head, eight partials' loads are in flight
// together, the first ones with their log-sum-exps'; the warps' sums meet in
// shared memory and are added in a fixed order.
// ---------------------------------------------------------------------------
template <typename T, int HD>
__global__ void __launch_bounds__(kMergeThreads) decode_merge_kernel(const KParams p) {
  constexpr int EL = HD / 32;  // elements per lane
  constexpr int NWARP = kMergeThreads / 32;
  __shared__ float red[NWARP][32][EL + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int W = p.merge_w, item = warp / W, sub = warp - item * W;
  const int64_t u = static_cast<int64_t>(blockIdx.x) * (NWARP / W) + item;
  // The W warps of an item decide together; no warp leaves before the CTA
  // barrier below (merge_w, and so the barrier, is the same for every CTA).
  int b = 0, hq = 0, c0 = 0, parts = 0, NC = 0, cb0 = 0, cb1 = 0;
  bool active = u < static_cast<int64_t>(p.B) * p.Hq;
  if (active) {
    b = static_cast<int>(u / p.Hq);
    hq = static_cast<int>(u - static_cast<int64_t>(b) * p.Hq);
  }
  if (p.inline_plan) {
    // the plan's sums anew, from the lengths: while the decode grid still runs
    const int cap = static_cast<int>(min(static_cast<int64_t>(p.max_ctx), static_cast<int64_t>(p.maxp) << p.log2P));
    int below = 0;
    for (int i = lane; i < p.B; i += 32) {
      const int L = p.ctx[i];
      const int n = L >= 1 && L <= cap ? (L + (1 << p.log2T) - 1) >> p.log2T : 0;
      NC += n;
      below += i < b ? n : 0;
      cb1 += i <= b ? n : 0;
    }
    NC = __reduce_add_sync(0xffffffffu, NC);
    cb0 = __reduce_add_sync(0xffffffffu, below);
    cb1 = __reduce_add_sync(0xffffffffu, cb1);
    pdl_wait();  // every partial of the decode grid is written
  } else {
    pdl_wait();
    NC = p.cs[p.B];
    cb0 = p.cs[b];
    cb1 = p.cs[b + 1];
  }
  if (cb1 <= cb0) active = false;
  if (active) {
    c0 = static_cast<int>(((static_cast<int64_t>(cb0) + 1) * p.n_ctas + NC - 1) / NC) - 1;
    const int c1 = static_cast<int>(((static_cast<int64_t>(cb1)) * p.n_ctas + NC - 1) / NC) - 1;
    parts = c1 - c0 + 1;
    active = c0 != c1;  // one CTA wrote the request whole
  }
  // With more CTAs than chunks some CTAs between c0 and c1 own no chunk and
  // wrote no partial: only CTAs with a non-empty range take part.  With at
  // least as many chunks as CTAs every CTA has a range.
  const bool all_busy = NC >= p.n_ctas;
  auto start = [&](int c) { return (static_cast<int64_t>(c) * NC) / p.n_ctas; };
  auto busy = [&](int cc) { return all_busy || start(cc) < start(cc + 1); };
  auto lse_of = [&](int k) { return p.lse_part[(static_cast<int64_t>(c0 + k) + b) * p.Hq + hq]; };
  float acc[EL];
#pragma unroll
  for (int e = 0; e < EL; ++e) acc[e] = 0.f;
  float wsum = 0.f;
  if (active) {
    const int per = (parts + W - 1) / W;
    const int k_begin = sub * per, k_end = min(parts, k_begin + per);
    // the first partials' loads do not wait for the weights'
    float v[8][EL];
    auto load = [&](int k0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (k0 + i < k_end) {
          const int64_t slot = static_cast<int64_t>(c0 + k0 + i) + b;
          const float* src = p.o_part + (slot * p.Hq + hq) * HD + lane * EL;
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
    float M = -INFINITY;
    for (int k = lane; k < parts; k += 32)
      if (busy(c0 + k)) M = fmaxf(M, lse_of(k));
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (M != -INFINITY) {
      for (int k0 = k_begin; k0 < k_end; k0 += 8) {
        if (k0 != k_begin) load(k0);
        const int k = k0 + lane;
        const float w_mine = lane < 8 && k < k_end && busy(c0 + k) ? exp2f(lse_of(k) - M) : 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float w = __shfl_sync(0xffffffffu, w_mine, i);
          if (w != 0.f) {  // (an idle CTA wrote no partial)
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
  if constexpr (sizeof(T) == 2) {
    if constexpr (EL == 4) {
      *reinterpret_cast<uint2*>(p.out + e0 * 2) =
          make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
    } else {
      *reinterpret_cast<uint32_t*>(p.out + e0 * 2) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
    }
  } else {
    if constexpr (EL == 4) {
      *reinterpret_cast<float4*>(p.out + e0 * 4) = make_float4(acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv);
    } else {
      *reinterpret_cast<float2*>(p.out + e0 * 4) = make_float2(acc[0] * inv, acc[1] * inv);
    }
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
inline cudaLaunchConfig_t cluster_config(int ctas, int threads, size_t smem) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  return cfg;
}
inline cudaLaunchAttribute cluster_attribute(int cluster) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = cluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  return attr;
}

// CTAs of one kernel instance that fit on an SM, or (cluster > 1) clusters of
// that many CTAs that fit on the GPU; cached per (device, kernel, smem, cluster).
struct OccKey {
  int device;
  const void* fn;
  int threads;
  size_t smem;
  int cluster;
};
constexpr int kOccKeys = 256;
std::mutex g_occ_mu;
OccKey g_occ_keys[kOccKeys];
int g_occ_vals[kOccKeys];
int g_occ_n = 0;

inline cudaError_t ctas_per_sm(const DeviceInfo& di, const void* fn, int threads, size_t smem, int* out,
                               int cluster = 0) {
  {
    std::lock_guard<std::mutex> lk(g_occ_mu);
    for (int i = 0; i < g_occ_n; ++i) {
      const OccKey& k = g_occ_keys[i];
      if (k.device == di.device && k.fn == fn && k.threads == threads && k.smem == smem && k.cluster == cluster) {
        *out = g_occ_vals[i];
        return cudaSuccess;
      }
    }
  }
  // The attribute is per kernel, not per launch: raise it to the device's
  // opt-in maximum so every plan's shared-memory size fits.
  cudaError_t e =
      cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, di.max_smem_optin);
  if (e != cudaSuccess) return e;
  // Prefer the largest shared-memory carve-out so that several CTAs fit.
  e = cudaFuncSetAttribute(fn, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  if (e != cudaSuccess) return e;
  int n = 0;
  if (cluster > 1) {
    cudaLaunchConfig_t cfg = cluster_config(cluster, threads, smem);
    cudaLaunchAttribute attr = cluster_attribute(cluster);
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&n, fn, &cfg);
    if (e != cudaSuccess) return e;
  } else {
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, fn, threads, smem);
    if (e != cudaSuccess) return e;
    if (n < 1) return cudaErrorInvalidConfiguration;
  }
  std::lock_guard<std::mutex> lk(g_occ_mu);
  if (g_occ_n < kOccKeys) {
    g_occ_keys[g_occ_n] = {di.device, fn, threads, smem, cluster};
    g_occ_vals[g_occ_n] = n;
    ++g_occ_n;
  }
  *out = n;
  return cudaSuccess;
}

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Workspace of a plan of n_ctas partitions: prefix sums, first requests, and
// the partial results' log-sum-exps and outputs.
inline void decode_workspace_layout(const pa_cache_desc& d, int batch, DecodePlan* pl) {
  size_t w = 0;
  pl->ws_cs = w;
  w = align_up(w + static_cast<size_t>(batch + 1) * 4, 256);
  pl->ws_cta_seq = w;
  w = align_up(w + static_cast<size_t>(pl->n_ctas) * 4, 256);
  pl->ws_lse = w;
  const size_t slots = static_cast<size_t>(pl->n_ctas) + batch;
  w = align_up(w + slots * d.num_q_heads * 4, 256);
  pl->ws_o = w;
  w = align_up(w + slots * d.num_q_heads * d.head_dim * 4, 256);
  pl->ws_bytes = w;
}

// The kernel parameters of a planned decode over a cache of row_bytes a token.
inline KParams decode_params(const pa_cache_desc& d, const DecodePlan& pl, const DecodeArgs& a, int row_bytes) {
  char* ws = static_cast<char*>(a.workspace);
  KParams p{};
  p.q = static_cast<const char*>(a.q);
  p.k_cache = static_cast<const char*>(a.k_cache);
  p.v_cache = static_cast<const char*>(a.v_cache);
  p.bt = a.block_tables;
  p.ctx = a.context_lens;
  p.out = static_cast<char*>(a.out);
  p.o_part = reinterpret_cast<float*>(ws + pl.ws_o);
  p.lse_part = reinterpret_cast<float*>(ws + pl.ws_lse);
  p.cs = reinterpret_cast<int32_t*>(ws + pl.ws_cs);
  p.cta_seq = reinterpret_cast<int32_t*>(ws + pl.ws_cta_seq);
  p.err = a.err;
  p.num_pages = d.num_pages;
  p.B = a.batch;
  p.Hq = d.num_q_heads;
  p.Hkv = d.num_kv_heads;
  p.P = d.page_size;
  p.maxp = a.max_pages;
  p.max_ctx = a.max_context_len;
  p.n_ctas = pl.n_ctas;
  p.log2P = 0;
  while ((1 << p.log2P) < d.page_size) ++p.log2P;
  p.log2T = 0;
  while ((1 << p.log2T) < pl.tokens_per_chunk) ++p.log2T;
  p.row_bytes = row_bytes;
  p.row_pitch = pl.row_pitch;
  p.chunk_bytes = pl.chunk_bytes;
  p.off_bar = pl.off_bar;
  p.off_meta = pl.off_meta;
  p.off_p = pl.off_p;
  p.off_alpha = pl.off_alpha;
  p.off_ml = pl.off_ml;
  p.off_abort = pl.off_abort;
  p.off_cs = pl.off_cs;
  p.inline_plan = a.batch <= kInlinePlanMax ? 1 : 0;
  p.p_row = pl.p_row;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.k_new = static_cast<const char*>(a.k_new);
  p.v_new = static_cast<const char*>(a.v_new);
  p.k_new_stride = a.k_new_stride_bytes;
  p.v_new_stride = a.v_new_stride_bytes;
  p.slot_out = a.slot_out;
  return p;
}

// Launches a planned decode: main_fn (whose arguments are main_args) between
// the plan kernel, where one is needed, and the merge.
inline cudaError_t launch_decode_kernels(const void* main_fn, const void* merge_fn, const DecodePlan& pl, KParams& p,
                                         void** main_args, cudaStream_t s) {
  // (plan ->) decode -> merge.  Up to kInlinePlanMax requests every decode CTA
  // computes the plan's prefix sums itself, which costs less than a kernel
  // boundary on the step's critical path; beyond, a plan kernel runs first.
  // The kernels after the first are launched to overlap their launch with the
  // kernel before them (each waits for it before reading its output).
  cudaError_t e;
  if (pl.cluster > 1) {
    cudaLaunchConfig_t cfg = cluster_config(pl.n_ctas, (pl.nw + 1) * 32, pl.smem_bytes);
    cfg.stream = s;
    cudaLaunchAttribute attr = cluster_attribute(pl.cluster);
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelExC(&cfg, main_fn, main_args);
  } else if (p.inline_plan) {
    e = cudaLaunchKernel(main_fn, dim3(pl.n_ctas), dim3((pl.nw + 1) * 32), main_args, pl.smem_bytes, s);
  } else {
    decode_plan_kernel<<<1, kPlanThreads, 0, s>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    e = launch_after_previous(main_fn, dim3(pl.n_ctas), dim3((pl.nw + 1) * 32), pl.smem_bytes, s, main_args);
  }
  if (e != cudaSuccess) return e;
  if (pl.n_ctas > 1 && pl.cluster == 0) {
    // warps per (request, q-head): about one per 8 partials of a request when
    // the requests are equally long (CTAs per request / 8), at most 4
    const int per_req = pl.n_ctas / std::max(1, p.B);
    p.merge_w = per_req >= 32 ? 4 : per_req >= 16 ? 2 : 1;
    const int64_t pairs = static_cast<int64_t>(p.B) * p.Hq;
    const int items = kMergeThreads / 32 / p.merge_w;
    const unsigned blocks = static_cast<unsigned>((pairs + items - 1) / items);
    void* args[] = {&p};
    e = launch_after_previous(merge_fn, dim3(blocks), dim3(kMergeThreads), 0, s, args);
    if (e != cudaSuccess) return e;
  }
  return cudaGetLastError();
}

}  // namespace
}  // namespace pa
