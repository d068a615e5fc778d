// Decode attention with a range of each request's keys left out (a sliding
// window with sinks; a prefix that the requests of a group share), and decode
// for such groups.  The kernel is decode_kernel.cuh's: the chunks wholly
// inside the range are not in a request's chunk list, so neither their pages
// nor the table entries that name them are read; the rows of the range in the
// chunks at its two ends are not copied (tensor-core consumers) and have
// probability 0.  Bytes per request: min(L, sinks + window) K and V rows; HBM
// bound like the kernel over all keys.
#include "decode_kernel.cuh"
#include "prefix_plan.cuh"

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

// ---------------------------------------------------------------------------
// Groups of requests that share a prefix.  Three kernels: the prefixes', whose
// tiles every query of a group meets at once (tcgen05 for bf16 with head_dim
// 128, else prefix_simt_kernel); the requests' own keys', beside it as its CTAs
// leave the SMs; the merge of both kernels' parts.
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
                        const float* lse_pre, int max_ctas) {
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
    const int ctas = prefix_ctas(s, total, max_ctas);
    const PrefixUnit unit = prefix_unit(s, gr, costs[g], h, (b - gr.s0) / s.TQ / 2);
    f0 = prefix_cta_of(unit.start, total, ctas);
    np = prefix_cta_of(unit.start + static_cast<int64_t>(gr.nt - 1) * unit.cost, total, ctas) - f0 + 1;
  }
  // the request's own: ns CTAs from c0 on
  int c0 = 0, ns = 0;
  if (cb1 > cb0) {
    c0 = static_cast<int>(((static_cast<int64_t>(cb0) + 1) * p.n_ctas + NC - 1) / NC) - 1;
    ns = static_cast<int>((static_cast<int64_t>(cb1) * p.n_ctas + NC - 1) / NC) - c0;
  }
  // without a prefix a single CTA's result is the output already
  active = active && (np > 0 || ns > 1);
  const int parts = np + ns;
  // with more CTAs than chunks, a CTA between the ends may have had none and left no part
  auto has = [&](int k) {
    if (k < np || NC >= p.n_ctas) return true;
    const int64_t c = c0 + k - np;
    return c * NC / p.n_ctas < (c + 1) * NC / p.n_ctas;
  };
  const int64_t pre_row = np > 0 ? prefix_part_row(gr.s0, gr.n, h, f0, p.Hq, G) + (b - gr.s0) * G + hq - h * G : 0;
  const int64_t own_row = static_cast<int64_t>(c0 + b) * p.Hq + hq;
  auto row_of = [&](int k) { return k < np ? pre_row + static_cast<int64_t>(k) * kPrefixPartRows
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
    const float lse_mine = lane < parts && has(lane) ? lse_of(lane) : -INFINITY;
    float M = lse_mine;
    for (int k = lane + 32; k < parts; k += 32)
      if (has(k)) M = fmaxf(M, lse_of(k));
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (M != -INFINITY) {
      const float w_first = exp2f(lse_mine - M);
      for (int k0 = k_begin; k0 < k_end; k0 += 8) {
        if (k0 != k_begin) load(k0);
        const int k = k0 + lane;
        float w_mine = 0.f;
        if (parts > 32 && lane < 8 && k < k_end && has(k)) w_mine = exp2f(lse_of(k) - M);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float w = parts > 32 ? __shfl_sync(0xffffffffu, w_mine, i)
                                     : __shfl_sync(0xffffffffu, w_first, (k0 + i) & 31);
          if (k0 + i < k_end && w != 0.f) {  // (an idle CTA wrote no part)
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

// ---------------------------------------------------------------------------
// attention to the prefixes on the CUDA cores (fp32, head_dim 64)
// ---------------------------------------------------------------------------
constexpr int kSimtThreads = 256, kSimtRows = 32;  // a warp has four rows of the unit

struct PrefixSimtParams {
  const char* q;
  const char* k_cache;
  const char* v_cache;
  const int32_t* bt;
  float* o_part;
  float* lse_part;
  unsigned int* err;
  int64_t* costs;
  PrefixShape shape;
  int64_t num_pages;
  int32_t Hq, G, maxp, log2P;
  float scale_log2;
};

template <int HD>
constexpr int kSimtFloats = kSimtRows * HD + kPrefixTile * (HD + 4) + kPrefixTile * HD + kSimtRows * kPrefixTile;
template <int HD>
constexpr int kSimtSmem = kSimtFloats<HD> * 4 + 64;  // and the unit at work

// A unit's rows stay in shared memory, the tile's K and V rows are brought there
// as fp32; a warp computes four rows against 128 keys (a lane four keys), their
// softmax by shuffles, and adds p V to its lanes' dims.
template <typename T, int HD>
__global__ void __launch_bounds__(kSimtThreads) prefix_simt_kernel(const PrefixSimtParams p) {
  extern __shared__ float4 simt_smem[];
  constexpr int E = sizeof(T), PER = 16 / E;  // elements of a 16-byte load
  constexpr int KP = HD + 4;                  // K row pitch: lanes' rows in different banks
  constexpr int DL = HD / 32;                 // dims a lane adds up
  float* qs = reinterpret_cast<float*>(simt_smem);
  float* ks = qs + kSimtRows * HD;
  float* vs = ks + kPrefixTile * KP;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  float* ps = vs + kPrefixTile * HD + warp * 4 * kPrefixTile;
  PrefixWork& work = *reinterpret_cast<PrefixWork*>(qs + kSimtFloats<HD>);
  int& more = *reinterpret_cast<int*>(&work + 1);
  static_assert(sizeof(PrefixWork) + sizeof(int) <= 64, "the unit at work and the flag fit");
  const int64_t row_bytes = static_cast<int64_t>(p.shape.Hkv) * HD * E;
  pdl_trigger();  // the decode kernel over the requests' own keys may start
  PrefixShare share;
  if (warp == 0) share = prefix_share(p.shape, blockIdx.x, gridDim.x, p.costs);
  for (;;) {
    if (tid == 0) {
      PrefixWork w;
      more = next_prefix_work(p.shape, share, w);
      work = w;
    }
    cta_sync();
    if (!more) return;
    const PrefixWork w = work;
    const int t0 = 2 * w.qp * p.shape.TQ;  // the unit's first request in its group
    const int rows = min(2 * p.shape.TQ, w.n - t0) * p.G;
    for (int i = tid; i < kSimtRows * HD / PER; i += kSimtThreads) {
      const int r = i / (HD / PER), d = i % (HD / PER) * PER;
      float f[PER];
#pragma unroll
      for (int e = 0; e < PER; ++e) f[e] = 0.f;
      if (r < rows) {
        const int64_t at = ((static_cast<int64_t>(w.s0) + t0 + r / p.G) * p.Hq + w.h * p.G + r % p.G) * HD + d;
        const T* src = reinterpret_cast<const T*>(p.q) + at;
#pragma unroll
        for (int e = 0; e < PER; ++e) f[e] = static_cast<float>(src[e]) * p.scale_log2;
      }
#pragma unroll
      for (int e = 0; e < PER; ++e) qs[r * HD + d + e] = f[e];
    }
    float m[4], l[4], o[4][DL];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
#pragma unroll
      for (int e = 0; e < DL; ++e) o[r][e] = 0.f;
    }
    const int32_t* table = p.bt + static_cast<int64_t>(w.rep) * p.maxp;
    for (int j = w.j_lo; j < w.j_hi; ++j) {
      const int key0 = j * kPrefixTile, keys = min(kPrefixTile, w.prefix - key0);
      cta_sync();  // the tile before has been read (and the queries are written)
      int bad = 0;
      for (int i = tid; i < kPrefixTile * HD / PER; i += kSimtThreads) {
        const int r = i / (HD / PER), d = i % (HD / PER) * PER;
        uint4 kw = make_uint4(0, 0, 0, 0), vw = kw;
        if (r < keys) {
          const int page = table[(key0 + r) >> p.log2P];
          if (page >= 0 && page < p.num_pages) {
            const int64_t slot = (static_cast<int64_t>(page) << p.log2P) + ((key0 + r) & ((1 << p.log2P) - 1));
            const int64_t at = slot * row_bytes + (w.h * HD + d) * E;
            kw = ldg16(p.k_cache + at);
            vw = ldg16(p.v_cache + at);
          } else {
            bad = 1;
          }
        }
        float kf[PER], vf[PER];
        if constexpr (E == 2) {
          const uint32_t a[4] = {kw.x, kw.y, kw.z, kw.w}, c[4] = {vw.x, vw.y, vw.z, vw.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 x = bf16x2_to_float2(a[e]), y = bf16x2_to_float2(c[e]);
            kf[2 * e] = x.x, kf[2 * e + 1] = x.y, vf[2 * e] = y.x, vf[2 * e + 1] = y.y;
          }
        } else {
          kf[0] = __uint_as_float(kw.x), kf[1] = __uint_as_float(kw.y);
          kf[2] = __uint_as_float(kw.z), kf[3] = __uint_as_float(kw.w);
          vf[0] = __uint_as_float(vw.x), vf[1] = __uint_as_float(vw.y);
          vf[2] = __uint_as_float(vw.z), vf[3] = __uint_as_float(vw.w);
        }
#pragma unroll
        for (int e = 0; e < PER; e += 4) {
          *reinterpret_cast<float4*>(ks + r * KP + d + e) = make_float4(kf[e], kf[e + 1], kf[e + 2], kf[e + 3]);
          *reinterpret_cast<float4*>(vs + r * HD + d + e) = make_float4(vf[e], vf[e + 1], vf[e + 2], vf[e + 3]);
        }
      }
      if (bad) raise_flag(p.err, PA_DEVERR_BAD_PAGE);
      cta_sync();
      if (4 * warp >= rows) continue;
      float2 acc[4][4];  // [row][key]: sums over even and odd dims
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[r][k] = make_float2(0.f, 0.f);
#pragma unroll 4
      for (int d = 0; d < HD; d += 4) {
        float4 kv[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) kv[k] = *reinterpret_cast<const float4*>(ks + (lane + 32 * k) * KP + d);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float4 qv = *reinterpret_cast<const float4*>(qs + (4 * warp + r) * HD + d);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            acc[r][k] = ffma2(make_float2(qv.x, qv.y), make_float2(kv[k].x, kv[k].y), acc[r][k]);
            acc[r][k] = ffma2(make_float2(qv.z, qv.w), make_float2(kv[k].z, kv[k].w), acc[r][k]);
          }
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float sc[4], mx = -INFINITY;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          sc[k] = lane + 32 * k < keys ? acc[r][k].x + acc[r][k].y : -INFINITY;
          mx = fmaxf(mx, sc[k]);
        }
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        const float m_new = fmaxf(m[r], mx), m_use = m_new == -INFINITY ? 0.f : m_new;
        const float alpha = exp2f(m[r] - m_use);
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float pv = exp2f(sc[k] - m_use);
          sum += pv;
          ps[r * kPrefixTile + lane + 32 * k] = pv;
        }
        l[r] = l[r] * alpha + sum;
        m[r] = m_new;
#pragma unroll
        for (int e = 0; e < DL; ++e) o[r][e] *= alpha;
      }
      __syncwarp();
      for (int k = 0; k < keys; k += 4) {
        float4 pr[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) pr[r] = *reinterpret_cast<const float4*>(ps + r * kPrefixTile + k);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {  // (rows past the last key are zero and have probability 0)
          float vf[DL];
          const float* src = vs + (k + kk) * HD + lane * DL;
#pragma unroll
          for (int e = 0; e < DL; ++e) vf[e] = src[e];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float pv = kk == 0 ? pr[r].x : kk == 1 ? pr[r].y : kk == 2 ? pr[r].z : pr[r].w;
#pragma unroll
            for (int e = 0; e < DL; ++e) o[r][e] = fmaf(pv, vf[e], o[r][e]);
          }
        }
      }
      __syncwarp();
    }
    const int64_t row0 = prefix_part_row(w.s0, w.n, w.h, blockIdx.x, p.Hq, p.G) + t0 * p.G;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], off);
      const int row = 4 * warp + r;
      if (row >= rows) continue;
      const float inv = l[r] > 0.f ? 1.f / l[r] : 0.f;
#pragma unroll
      for (int e = 0; e < DL; ++e) p.o_part[(row0 + row) * HD + lane * DL + e] = o[r][e] * inv;
      if (lane == 0) p.lse_part[row0 + row] = l[r] > 0.f ? m[r] + log2f(l[r]) : -INFINITY;
    }
  }
}

bool prefix_on_tensor_cores(const pa_cache_desc& d) { return d.dtype == PA_BF16 && d.head_dim == 128; }

template <typename T, int HD>
cudaError_t launch_prefix_simt(const pa_cache_desc& d, const SharedArgs& a, const SharedPlan& pl, cudaStream_t s) {
  DeviceInfo di;
  cudaError_t e = current_device_info(&di);
  if (e != cudaSuccess) return e;
  const void* fn = reinterpret_cast<const void*>(prefix_simt_kernel<T, HD>);
  int occ = 0;  // (sets the kernel's shared-memory attributes)
  if ((e = ctas_per_sm(di, fn, kSimtThreads, kSimtSmem<HD>, &occ)) != cudaSuccess) return e;
  char* ws = static_cast<char*>(a.workspace);
  PrefixSimtParams p{};
  p.q = static_cast<const char*>(a.q);
  p.k_cache = static_cast<const char*>(a.k_cache);
  p.v_cache = static_cast<const char*>(a.v_cache);
  p.bt = a.block_tables;
  p.o_part = reinterpret_cast<float*>(ws + pl.off_o);
  p.lse_part = reinterpret_cast<float*>(ws + pl.off_lse);
  p.err = a.err;
  p.shape = prefix_shape(d, a, pl);
  p.costs = reinterpret_cast<int64_t*>(ws + pl.off_costs);
  p.num_pages = d.num_pages;
  p.Hq = d.num_q_heads;
  p.G = d.num_q_heads / d.num_kv_heads;
  p.maxp = a.max_pages;
  while ((1 << p.log2P) < d.page_size) ++p.log2P;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  prefix_simt_kernel<T, HD><<<pl.prefix_ctas, kSimtThreads, kSimtSmem<HD>, s>>>(p);
  return cudaGetLastError();
}

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
  return s;
}

cudaError_t plan_shared(const pa_cache_desc& d, int n_groups, int batch, int max_prefix, int max_ctx, int max_ctas,
                        SharedPlan* out) {
  SharedPlan pl;
  cudaError_t e = plan_decode_keys<true>(d, batch, max_ctx, 0, max_ctas, &pl.suffix);
  if (e != cudaSuccess) return e;
  pl.ws_bytes = align_up(pl.suffix.ws_bytes, 256);
  if (n_groups > 0 && max_prefix > 0) {
    DeviceInfo di;
    if ((e = current_device_info(&di)) != cudaSuccess) return e;
    const int G = d.num_q_heads / d.num_kv_heads;
    const bool tc = prefix_on_tensor_cores(d);
    pl.prefix_ctas = max_ctas > 0 ? std::min(max_ctas, di.sm_count) : di.sm_count;
    pl.TQ = (tc ? 128 : kSimtRows / 2) / G;
    // a tile of one q-tile alone takes about 0.7 of the time that one of two takes
    pl.cost_pair = tc ? 10 : 1;
    pl.cost_one = tc ? 7 : 1;
    const int64_t rows = static_cast<int64_t>(batch) * d.num_q_heads + static_cast<int64_t>(pl.prefix_ctas) * 256;
    if (rows >= int64_t(1) << 31) return cudaErrorInvalidValue;
    // TMA coordinates are 32-bit: the cache rows must be addressable
    if (tc && d.num_pages * d.page_size >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
    pl.off_costs = pl.ws_bytes;
    pl.off_lse = align_up(pl.off_costs + (static_cast<size_t>(n_groups) + 1) * 8, 256);
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
  const Fns f = get_fns<true>(d.dtype, d.head_dim, d.num_q_heads / d.num_kv_heads);
  if (!f.main) return cudaErrorInvalidValue;
  KParams p = decode_params(d, pl.suffix, da, d.num_kv_heads * d.head_dim * elem_bytes(d.dtype));
  void* args[] = {&p};
  if (pl.prefix_ctas == 0) {  // no prefixes: plain decode (a window of everything)
    p.window = a.max_context_len;
    return launch_decode_kernels<true>(f.main, f.merge, pl.suffix, p, args, s);
  }
  p.cu_groups = a.cu_groups;
  p.prefix_lens = a.prefix_lens;
  p.n_groups = a.n_groups;
  p.max_prefix = a.max_prefix;
  cudaError_t e;
  if (prefix_on_tensor_cores(d))
    e = launch_prefix_tc(d, a, pl, s);
  else if (d.dtype == PA_BF16)
    e = launch_prefix_simt<__nv_bfloat16, 64>(d, a, pl, s);
  else
    e = d.head_dim == 128 ? launch_prefix_simt<float, 128>(d, a, pl, s) : launch_prefix_simt<float, 64>(d, a, pl, s);
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
  int max_ctas = pl.prefix_ctas;
  void* margs[] = {&p, &shape, &costs, &o_pre, &lse_pre, &max_ctas};
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
