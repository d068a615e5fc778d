// Writing rows into a 4-bit cache and reading them back (sm_103a).
//
// Both are one pass over the data and HBM-bound: writing a token reads
// 2 * Hkv * HD elements and writes 2 rows of (HD / 2 + 4 HD / GS) * Hkv bytes,
// reading does the reverse.
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
// write: a thread takes eight dims of one (token, kv-head), K and V
// ---------------------------------------------------------------------------
template <typename T, int HD, int GS>
__global__ void __launch_bounds__(kQ4Threads) kv_write_q4_kernel(const Q4WriteParams p) {
  constexpr int LPR = HD / 8;   // lanes per head row
  constexpr int NG = HD / GS;   // groups per head row
  pdl_trigger();                // as in kv_write_kernel
  const uint32_t per_tok = static_cast<uint32_t>(p.hkv) * LPR;
  const uint32_t codes = static_cast<uint32_t>(p.hkv) * (HD / 2), pars = static_cast<uint32_t>(p.row_bytes) - codes;
  const int64_t total = p.n_tokens * per_tok;
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  // whole warps go round together (the groups' reductions are warp shuffles)
  for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * blockDim.x + (threadIdx.x & ~31u); i0 < total; i0 += step) {
    const int64_t i = i0 + (threadIdx.x & 31u);
    const int64_t t = i / per_tok;
    const uint32_t r = static_cast<uint32_t>(i - t * per_tok), h = r / LPR, l = r % LPR;
    int64_t slot = -1;
    if (i < total) {
      slot = p.slots[t];
      if (slot < 0 || slot >= p.num_slots) {
        if (slot != -1 && r == 0) raise_flag(p.err, PA_DEVERR_BAD_SLOT);
        slot = -1;
      }
    }
    float k[8] = {}, v[8] = {};
    if (slot >= 0) {
      q4_load8<T>(p.k + t * p.k_stride_bytes + r * (8 * sizeof(T)), k);
      q4_load8<T>(p.v + t * p.v_stride_bytes + r * (8 * sizeof(T)), v);
    }
    uint32_t kp, vp;
    const uint32_t kw = q4_quantise8(k, GS / 8, kp), vw = q4_quantise8(v, GS / 8, vp);
    if (slot >= 0) {
      const uint32_t tt = static_cast<uint32_t>(slot);
      const uint32_t co = q4_swz(r * 4, codes, tt);
      char* kr = p.k_cache + slot * p.row_bytes;
      char* vr = p.v_cache + slot * p.row_bytes;
      *reinterpret_cast<uint32_t*>(kr + co) = kw;
      *reinterpret_cast<uint32_t*>(vr + co) = vw;
      if (l % (GS / 8) == 0) {
        const uint32_t po = codes + q4_swz((h * NG + l / (GS / 8)) * 4, pars, tt);
        *reinterpret_cast<uint32_t*>(kr + po) = kp;
        *reinterpret_cast<uint32_t*>(vr + po) = vp;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// read back: a CTA takes kReadRows consecutive output rows; their slots are
// looked up first (one thread a row), then a thread takes eight dims of a row
// ---------------------------------------------------------------------------
constexpr int kReadRows = 16;

template <typename T, int HD, int GS>
__global__ void __launch_bounds__(kQ4Threads) kv_read_q4_kernel(const Q4ReadParams p) {
  constexpr int LPR = HD / 8;
  constexpr int NG = HD / GS;
  __shared__ int64_t slot_s[kReadRows];
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kReadRows;
  const int rows = static_cast<int>(min(static_cast<int64_t>(kReadRows), p.num_rows - row0));
  if (threadIdx.x < rows) {
    const int64_t r = row0 + threadIdx.x;
    int lo = 0, hi = p.batch - 1;  // the last request whose rows start at or before r
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
  const uint32_t per_row = static_cast<uint32_t>(p.hkv) * LPR;
  const uint32_t codes = static_cast<uint32_t>(p.hkv) * (HD / 2), pars = static_cast<uint32_t>(p.row_bytes) - codes;
  const uint32_t total = rows * per_row;
#pragma unroll 4
  for (uint32_t i = threadIdx.x; i < total; i += kQ4Threads) {
    const uint32_t rr = i / per_row, r = i - rr * per_row, h = r / LPR, l = r % LPR;
    const int64_t slot = slot_s[rr];
    if (slot < 0) continue;
    const uint32_t tt = static_cast<uint32_t>(slot);
    const uint32_t co = q4_swz(r * 4, codes, tt);
    const uint32_t po = codes + q4_swz((h * NG + l / (GS / 8)) * 4, pars, tt);
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      const char* src = (part ? p.v_cache : p.k_cache) + slot * p.row_bytes;
      const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(src + co));
      const float2 sc = q4_sc(__ldg(reinterpret_cast<const uint32_t*>(src + po)));
      float a[4], b[4];
      q4_decode4(w & 0xFFFFu, sc.x, sc.y, a);
      q4_decode4(w >> 16, sc.x, sc.y, b);
      const float x[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
      char* dst = part ? p.v_out + (row0 + rr) * p.v_stride_bytes : p.k_out + (row0 + rr) * p.k_stride_bytes;
      store8<T>(dst + r * (8 * sizeof(T)), x);
    }
  }
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
  const int64_t total = p.n_tokens * p.hkv * (d.head_dim / 8);
  const int64_t blocks =
      std::min<int64_t>((total + kQ4Threads - 1) / kQ4Threads, static_cast<int64_t>(di.sm_count) * 8);
  void* args[] = {const_cast<Q4WriteParams*>(&p)};
  e = cudaLaunchKernel(fn, dim3(static_cast<unsigned>(blocks)), dim3(kQ4Threads), args, 0, s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_kv_read_q4(const pa_cache_desc& d, int gs, const Q4ReadParams& p, cudaStream_t s) {
  const void* fn = d.dtype == PA_BF16
                       ? (d.head_dim == 128 ? read_fn<__nv_bfloat16, 128>(gs) : read_fn<__nv_bfloat16, 64>(gs))
                       : (d.head_dim == 128 ? read_fn<float, 128>(gs) : read_fn<float, 64>(gs));
  const unsigned blocks = static_cast<unsigned>((p.num_rows + kReadRows - 1) / kReadRows);
  void* args[] = {const_cast<Q4ReadParams*>(&p)};
  cudaError_t e = cudaLaunchKernel(fn, dim3(blocks), dim3(kQ4Threads), args, 0, s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace pa
