// Writing rows into a 4-bit cache and reading them back (sm_103a).
//
// Both are one pass over the data: writing a token reads 2 * Hkv * HD elements and
// writes 2 rows of (HD / 2 + 4 HD / GS) * Hkv bytes, reading does the reverse.
// Measured (8 heads of 128 dims, bf16): writing 16384 tokens 22.4 us, 3.9 TB/s,
// bound by its 1043 warp instructions a token (72% issue active) once K and V share
// the work on their groups' parameters; reading 32768 rows 31 us and 89554 rows
// 74.3 us, 5.5 and 6.2 TB/s of a copy's 6.7.
#include <algorithm>

#include "q4_common.cuh"

namespace pa {
namespace {

constexpr int kQ4Threads = 256;

template <typename T>
PA_DEVINL void store8(char* p, const float (&x)[8]) {
  if constexpr (sizeof(T) == 2) {
    stg16(p, make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                        pack_bf16x2(x[6], x[7])));
  } else {
    stg16(p, make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])));
    stg16(p + 16,
          make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7])));
  }
}

// ---------------------------------------------------------------------------
// write: a thread takes eight dims of one kv-head, K and V, of every kQ4Threads /
// (threads of a token)-th token; the loads of two tokens are in flight together
// ---------------------------------------------------------------------------
template <typename T, int HD, int GS>
__global__ void __launch_bounds__(kQ4Threads) kv_write_q4_kernel(const Q4WriteParams p) {
  pdl_trigger();                // as in kv_write_kernel
  const uint32_t per_tok = static_cast<uint32_t>(p.hkv) * (HD / 8);  // threads of a token: a power of two, 8 to 128
  const uint32_t codes = static_cast<uint32_t>(p.hkv) * (HD / 2), pars = static_cast<uint32_t>(p.row_bytes) - codes;
  const uint32_t r = threadIdx.x & (per_tok - 1);
  const uint32_t sub = threadIdx.x >> (31 - __clz(per_tok)), tpc = kQ4Threads >> (31 - __clz(per_tok));  // tokens per CTA
  const uint32_t co = r * 4, po = r / (GS / 8) * 4;
  const bool leads = r % (GS / 8) == 0;  // stores its group's parameters
  const int64_t step = static_cast<int64_t>(gridDim.x) * tpc;
  // whole CTAs go round together (the groups' reductions are warp shuffles)
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * tpc; t0 < p.n_tokens; t0 += 2 * step) {
    uint32_t kw[2][kQ4Words<T>], vw[2][kQ4Words<T>];
    int64_t slot[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int64_t t = t0 + u * step + sub;
      slot[u] = -1;
      if (t < p.n_tokens) {
        slot[u] = p.slots[t];
        if (slot[u] < 0 || slot[u] >= p.num_slots) {
          if (slot[u] != -1 && r == 0) raise_flag(p.err, PA_DEVERR_BAD_SLOT);
          slot[u] = -1;
        }
        // a token that is not stored is read all the same: its loads need not wait for its slot
        q4_load8<T>(p.k + t * p.k_stride_bytes + r * (8 * sizeof(T)), kw[u]);
        q4_load8<T>(p.v + t * p.v_stride_bytes + r * (8 * sizeof(T)), vw[u]);
      } else {
#pragma unroll
        for (int e = 0; e < kQ4Words<T>; ++e) kw[u][e] = vw[u][e] = 0u;
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (u == 1 && t0 + step >= p.n_tokens) break;  // the same for the whole CTA
      uint32_t kp, vp, kc, vc;
      q4_quantise8_pair<T>(kw[u], vw[u], GS / 8, kc, vc, kp, vp);
      if (slot[u] >= 0) {
        const uint32_t tt = static_cast<uint32_t>(slot[u]);
        char* kr = p.k_cache + slot[u] * p.row_bytes;
        char* vr = p.v_cache + slot[u] * p.row_bytes;
        *reinterpret_cast<uint32_t*>(kr + q4_swz(co, codes, tt)) = kc;
        *reinterpret_cast<uint32_t*>(vr + q4_swz(co, codes, tt)) = vc;
        if (leads) {
          *reinterpret_cast<uint32_t*>(kr + codes + q4_swz(po, pars, tt)) = kp;
          *reinterpret_cast<uint32_t*>(vr + codes + q4_swz(po, pars, tt)) = vp;
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// read back: a CTA takes `rows_per_cta` consecutive output rows.  Their slots are
// looked up first; then a thread takes eight dims of every row of its share, the
// loads of kReadRows rows in flight together.
// ---------------------------------------------------------------------------
constexpr int kMaxReadRows = kQ4Threads;  // a thread looks up one row
constexpr int kReadRows = 4;

// The number of requests whose rows start at or before row r, by the whole CTA.
PA_DEVINL int requests_from(const Q4ReadParams& p, int64_t r) {
  int n = 0;
  for (int b0 = 0; b0 < p.batch; b0 += kQ4Threads) {
    const int b = b0 + static_cast<int>(threadIdx.x);
    n += __syncthreads_count(b < p.batch && p.cu[b] <= r);
  }
  return n;
}

template <typename T, int HD, int GS>
__global__ void __launch_bounds__(kQ4Threads) kv_read_q4_kernel(const Q4ReadParams p) {
  __shared__ int64_t slot_s[kMaxReadRows];
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * p.rows_per_cta;
  const int rows = static_cast<int>(min(static_cast<int64_t>(p.rows_per_cta), p.num_rows - row0));
  // requests of the first and the last row (cu_rows does not fall), then each row's between them
  const int first = max(requests_from(p, row0) - 1, 0), last = max(requests_from(p, row0 + rows - 1) - 1, first);
  if (threadIdx.x < rows) {
    const int64_t r = row0 + threadIdx.x;
    int lo = first, hi = last;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (p.cu[mid] <= r) lo = mid;
      else hi = mid - 1;
    }
    const int s0 = p.cu[lo], s1 = p.cu[lo + 1], L = p.ctx[lo], start = p.starts ? p.starts[lo] : 0;
    int64_t slot = -1;
    unsigned int flag = 0;
    if (r >= s1 && lo == p.batch - 1) {
      // past the last request's rows
    } else if (s0 < 0 || r < s0 || r >= s1) {
      flag = PA_DEVERR_BAD_LENGTH;  // cu_rows does not cover the row
    } else if (L == 0) {
      // a padding request
    } else if (L < 0 || start < 0 || static_cast<int64_t>(L) > static_cast<int64_t>(p.maxp) << p.log2P) {
      flag = PA_DEVERR_BAD_LENGTH;
    } else {
      const int64_t pos = start + (r - s0);
      if (pos < L) {
        const int page = p.bt[static_cast<int64_t>(lo) * p.maxp + (pos >> p.log2P)];
        if (page >= 0 && page < p.num_pages)
          slot = (static_cast<int64_t>(page) << p.log2P) + (pos & ((1 << p.log2P) - 1));
        else
          flag = PA_DEVERR_BAD_PAGE;
      }
    }
    if (flag) raise_flag(p.err, flag);
    slot_s[threadIdx.x] = slot;
  }
  cta_sync();
  const uint32_t per_row = static_cast<uint32_t>(p.hkv) * (HD / 8);  // threads of a row: a power of two, 8 to 128
  const uint32_t codes = static_cast<uint32_t>(p.hkv) * (HD / 2), pars = static_cast<uint32_t>(p.row_bytes) - codes;
  const uint32_t r = threadIdx.x & (per_row - 1);
  const int sub = threadIdx.x >> (31 - __clz(per_row)), step = kQ4Threads >> (31 - __clz(per_row));
  const uint32_t co = r * 4, po = r / (GS / 8) * 4;
  char* k_out = p.k_out + row0 * p.k_stride_bytes + r * (8 * sizeof(T));
  char* v_out = p.v_out + row0 * p.v_stride_bytes + r * (8 * sizeof(T));
  for (int r0 = sub; r0 < rows; r0 += kReadRows * step) {
    uint32_t w[kReadRows][2], sc[kReadRows][2];
    bool live[kReadRows];
#pragma unroll
    for (int u = 0; u < kReadRows; ++u) {
      const int rr = r0 + u * step;
      int64_t slot = rr < rows ? slot_s[rr] : -1;
      live[u] = slot >= 0;
      slot = max(slot, static_cast<int64_t>(0));  // (a row that is not read loads slot 0: no branch between the loads)
      const uint32_t tt = static_cast<uint32_t>(slot);
      const char* kr = p.k_cache + slot * p.row_bytes;
      const char* vr = p.v_cache + slot * p.row_bytes;
      const uint32_t c = q4_swz(co, codes, tt), q = codes + q4_swz(po, pars, tt);
      w[u][0] = __ldg(reinterpret_cast<const uint32_t*>(kr + c));
      w[u][1] = __ldg(reinterpret_cast<const uint32_t*>(vr + c));
      sc[u][0] = __ldg(reinterpret_cast<const uint32_t*>(kr + q));
      sc[u][1] = __ldg(reinterpret_cast<const uint32_t*>(vr + q));
    }
#pragma unroll
    for (int u = 0; u < kReadRows; ++u) {
      if (!live[u]) continue;
      const int64_t rr = r0 + u * step;
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        const float2 g = q4_sc(sc[u][part]);
        float x[8];
        q4_decode8(w[u][part], g.x, g.y, x);
        store8<T>(part ? v_out + rr * p.v_stride_bytes : k_out + rr * p.k_stride_bytes, x);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// block tables of the rows read back: a thread takes an entry
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kQ4Threads) kv_read_tables_kernel(const Q4TablesParams p) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kQ4Threads + threadIdx.x;
  if (i >= static_cast<int64_t>(p.batch) * p.maxp_out) return;
  const int b = static_cast<int>(i / p.maxp_out), j = static_cast<int>(i - static_cast<int64_t>(b) * p.maxp_out);
  const int first = p.cu[b], end = p.cu[b + 1];
  int page = -1;
  if (j < p.maxp && first >= 0 && first + (static_cast<int64_t>(j + 1) << p.log2P) <= end) {
    const int src = p.bt[static_cast<int64_t>(b) * p.maxp + j];
    if (src >= 0 && src < p.num_pages) page = (first >> p.log2P) + j;
  }
  p.out[i] = page;
}

template <typename T, int HD>
const void* write_fn(int gs) {
  if constexpr (HD == 128)
    if (gs == 128) return reinterpret_cast<const void*>(kv_write_q4_kernel<T, HD, 128>);
  return gs == 64 ? reinterpret_cast<const void*>(kv_write_q4_kernel<T, HD, 64>)
                  : reinterpret_cast<const void*>(kv_write_q4_kernel<T, HD, 32>);
}

template <typename T, int HD>
const void* read_fn(int gs) {
  if constexpr (HD == 128)
    if (gs == 128) return reinterpret_cast<const void*>(kv_read_q4_kernel<T, HD, 128>);
  return gs == 64 ? reinterpret_cast<const void*>(kv_read_q4_kernel<T, HD, 64>)
                  : reinterpret_cast<const void*>(kv_read_q4_kernel<T, HD, 32>);
}

}  // namespace

cudaError_t launch_kv_write_q4(const pa_cache_desc& d, int gs, const Q4WriteParams& p, cudaStream_t s) {
  DeviceInfo di;
  cudaError_t e = current_device_info(&di);
  if (e != cudaSuccess) return e;
  const void* fn = d.dtype == PA_BF16
                       ? (d.head_dim == 128 ? write_fn<__nv_bfloat16, 128>(gs) : write_fn<__nv_bfloat16, 64>(gs))
                       : (d.head_dim == 128 ? write_fn<float, 128>(gs) : write_fn<float, 64>(gs));
  const int tpc = kQ4Threads / (p.hkv * (d.head_dim / 8));  // tokens a CTA takes at a time
  const int64_t blocks = std::min<int64_t>((p.n_tokens + tpc - 1) / tpc, static_cast<int64_t>(di.sm_count) * 8);
  void* args[] = {const_cast<Q4WriteParams*>(&p)};
  e = cudaLaunchKernel(fn, dim3(static_cast<unsigned>(blocks)), dim3(kQ4Threads), args, 0, s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_kv_read_tables(const Q4TablesParams& p, cudaStream_t s) {
  const int64_t n = static_cast<int64_t>(p.batch) * p.maxp_out;
  const int64_t blocks = (n + kQ4Threads - 1) / kQ4Threads;  // (below 2^31: the caller's check)
  kv_read_tables_kernel<<<static_cast<unsigned>(blocks), kQ4Threads, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_kv_read_q4(const pa_cache_desc& d, int gs, Q4ReadParams p, cudaStream_t s) {
  DeviceInfo di;
  cudaError_t e = current_device_info(&di);
  if (e != cudaSuccess) return e;
  const void* fn = d.dtype == PA_BF16
                       ? (d.head_dim == 128 ? read_fn<__nv_bfloat16, 128>(gs) : read_fn<__nv_bfloat16, 64>(gs))
                       : (d.head_dim == 128 ? read_fn<float, 128>(gs) : read_fn<float, 64>(gs));
  // Rows per CTA: what its threads take in one go (kReadRows each); twice that
  // where it still leaves 12 CTAs an SM (the look-up of the rows' slots, about
  // 2 us, is paid half as often: 89.6k rows 77.9 -> 74.6 us, but 16.4k rows
  // 18.8 -> 19.5 us); less where SMs would have no work.
  const int64_t at_once = kQ4Threads / (p.hkv * (d.head_dim / 8));
  int64_t rows = at_once * kReadRows;
  if (p.num_rows / (2 * rows) >= 12 * di.sm_count) rows *= 2;
  while (rows > at_once && p.num_rows / rows < 2 * di.sm_count) rows /= 2;
  p.rows_per_cta = static_cast<int32_t>(std::min<int64_t>(rows, kMaxReadRows));
  const unsigned blocks = static_cast<unsigned>((p.num_rows + p.rows_per_cta - 1) / p.rows_per_cta);
  void* args[] = {&p};
  e = cudaLaunchKernel(fn, dim3(blocks), dim3(kQ4Threads), args, 0, s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace pa
