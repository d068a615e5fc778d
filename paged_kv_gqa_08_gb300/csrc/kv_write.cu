// Slot mapping, KV scatter, and the fused per-head Q/K RMSNorm + RoPE + KV
// scatter (sm_103a).  All three are small, latency- or HBM-bound kernels.
#include <limits.h>
#include <math.h>

#include <algorithm>

#include "q4_common.cuh"

namespace pa {
namespace {

// ---------------------------------------------------------------------------
// slot mapping (nano-vLLM learning note, prepare_prefill / prepare_decode)
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(128) slot_mapping_kernel(const SlotMapParams p) {
  const int b = blockIdx.x;
  const int s0 = p.cu_seqlens_q[b], s1 = p.cu_seqlens_q[b + 1];
  const int L = p.context_lens[b];
  const int n = s1 - s0;
  const int start = L - n;
  if (L == 0 && n >= 0 && s0 >= 0 && static_cast<int64_t>(s1) <= p.num_tokens) {
    // A padding row (length 0: a batch padded up to a fixed size): its tokens
    // are stored nowhere.
    for (int j = threadIdx.x; j < n; j += blockDim.x) {
      p.positions[s0 + j] = 0;
      p.slots[s0 + j] = -1;
    }
    return;
  }
  const bool ok = n >= 0 && start >= 0 && s0 >= 0 && static_cast<int64_t>(s1) <= p.num_tokens &&
                  static_cast<int64_t>(L) <= static_cast<int64_t>(p.max_pages) * p.page_size;
  if (!ok) {
    if (threadIdx.x == 0) raise_flag(p.err, PA_DEVERR_BAD_LENGTH);
    // Leave well-formed rows of this request marked "store nothing".
    if (n > 0 && s0 >= 0 && static_cast<int64_t>(s1) <= p.num_tokens)
      for (int j = threadIdx.x; j < n; j += blockDim.x) {
        p.positions[s0 + j] = 0;
        p.slots[s0 + j] = -1;
      }
    return;
  }
  for (int j = threadIdx.x; j < n; j += blockDim.x) {
    const int pos = start + j;
    const int page = p.block_tables[static_cast<int64_t>(b) * p.max_pages + pos / p.page_size];
    int64_t slot = -1;
    if (page >= 0 && page < p.num_pages) {
      slot = static_cast<int64_t>(page) * p.page_size + pos % p.page_size;
    } else {
      raise_flag(p.err, PA_DEVERR_BAD_PAGE);
    }
    p.positions[s0 + j] = pos;
    p.slots[s0 + j] = slot;
  }
}

// ---------------------------------------------------------------------------
// KV scatter (nano-vLLM learning note, store_kvcache_kernel): 16-byte chunks,
// one thread per chunk of K and the same chunk of V.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) kv_write_kernel(const KvWriteParams p) {
  // the prefill planner of the same step may start beside this grid (it
  // reads none of its output and waits for it before it exits)
  pdl_trigger();
  const uint32_t cpr = static_cast<uint32_t>(p.row_bytes) >> 4;
  const int64_t total = p.n_tokens * cpr;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t t = i / cpr;
    const uint32_t ch = static_cast<uint32_t>(i - t * cpr);
    const int64_t slot = p.slots[t];
    if (slot < 0 || slot >= p.num_slots) {
      if (slot != -1 && ch == 0) raise_flag(p.err, PA_DEVERR_BAD_SLOT);
      continue;
    }
    const uint4 kw = ldg16(p.k + t * p.k_stride_bytes + ch * 16);
    const uint4 vw = ldg16(p.v + t * p.v_stride_bytes + ch * 16);
    stg16(p.k_cache + slot * p.row_bytes + ch * 16, kw);
    stg16(p.v_cache + slot * p.row_bytes + ch * 16, vw);
  }
}

// ---------------------------------------------------------------------------
// fused q/k RMSNorm + rotary + KV scatter.  One CTA (4 warps) per token.
// A group of LPH lanes handles one head: lane l owns elements
// [4l, 4l+4) of the first half and the same of the second half, so each lane
// holds both members of its rotation pairs.  Values are rounded to the storage
// type after the normalisation, after the weight and after the rotation (the
// casts of the Qwen3 norm and rotary in the nano-vLLM learning note); for bf16
// the element arithmetic runs on fp32 pairs (packed multiplies and FMAs, one
// two-lane conversion per rounding).
// ---------------------------------------------------------------------------
template <typename T>
struct Vec4;
template <>
struct Vec4<float> {
  static PA_DEVINL void load(const void* p, float (&x)[4]) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
  }
  static PA_DEVINL void store(void* p, const float (&x)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  }
};
template <>
struct Vec4<__nv_bfloat16> {
  static PA_DEVINL void load(const void* p, float (&x)[4]) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    const float2 a = bf16x2_to_float2(v.x), b = bf16x2_to_float2(v.y);
    x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
  }
  static PA_DEVINL void store(void* p, const float (&x)[4]) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
  }
};

PA_DEVINL void load_two(const float* p, float& x, float& y) {
  const float2 v = *reinterpret_cast<const float2*>(p);
  x = v.x;
  y = v.y;
}
PA_DEVINL void load_two(const __nv_bfloat16* p, float& x, float& y) {
  const float2 v = bf16x2_to_float2(*reinterpret_cast<const uint32_t*>(p));
  x = v.x;
  y = v.y;
}

// 2*pi as the float nearest to it plus the float nearest to the remainder
// (Cody and Waite's additive reduction, 1980), and the float nearest to 1/(2*pi).
constexpr float kTwoPiF1 = 6.28318548202514648f;
constexpr float kTwoPiF2 = -1.74845553146951609e-7f;
constexpr float kInvTwoPiF = 0.159154943091895336f;

// The rotation angle pos * f reduced into [-pi, pi], with f given as the float
// pair fh + fl.  pos * fh is split exactly into p1 + e1 (an FMA recovers the
// product's rounding error: Dekker's two-product); pos * fl is below 2^-24 of
// the angle, so one rounding of it is negligible.  The angle is then reduced
// by k = rint(pos * fh / (2 pi)) against the two-float 2 pi: each FMA's result
// is exact or within an ulp of a value below pi, so for angles up to ~2^17 rad
// (positions up to ~131k at frequency 1) the reduced angle is within a few
// 1e-7 rad of the exact one.
PA_DEVINL float reduce_angle(int pos, float fh, float fl) {
  const float pf = static_cast<float>(pos);  // exact below 2^24
  const float p1 = pf * fh;
  const float e1 = fmaf(pf, fh, -p1);
  const float e2 = pf * fl;
  const float k = rintf(p1 * kInvTwoPiF);
  const float r = fmaf(-k, kTwoPiF2, fmaf(-k, kTwoPiF1, p1));
  return r + (e1 + e2);
}

// a + b = s + e exactly (Knuth).
PA_DEVINL void two_sum(float a, float b, float& s, float& e) {
  s = a + b;
  const float bb = s - a;
  e = (a - (s - bb)) + (b - bb);
}

// Sine and cosine of pos * f, f = fh + fl but for 2^-49 of itself, rounded to fp32
// from about 2^-35 of their value (0.06% of them differ from the rounded double
// result, by one ulp).  The angle is a float pair, reduced by multiples of pi/2 in
// three floats (p - k C1 is exact: both are multiples of the result's last place).
// From position 2^17 on, where the pair's 2^-49 of the angle would begin to show (and
// 2^24, where a float no longer holds every position), angle and reduction are in 64
// bits.  The Taylor series' first correction (-r^3/6, r^4/24) is a float pair too, the
// rest of either series too small to need one.
PA_DEVINL void sincos_pair(int pos, float fh, float fl, double f, float& sn, float& cs) {
  float r, rl;
  int q;
  if (pos < 1 << 17) {
    const float pf = static_cast<float>(pos);
    const float p = __fmul_rn(pf, fh), lo = fmaf(pf, fl, fmaf(pf, fh, -p));
    const float k = rintf(p * 0.636619772f);
    const float h = __fmul_rn(k, -4.37113883e-8f), l = fmaf(k, -1.71512451e-15f, fmaf(k, -4.37113883e-8f, -h));
    float s1, e1, s2, e2;
    two_sum(fmaf(-k, 1.57079637f, p), lo, s1, e1);
    two_sum(s1, -h, s2, e2);
    two_sum(s2, (e1 + e2) - l, r, rl);
    q = static_cast<int>(k);
  } else {
    const double a = pos * f, k = rint(a * 0.63661977236758134);
    const double d = fma(-k, 6.123233995736766e-17, fma(-k, 1.5707963267948966, a));
    r = static_cast<float>(d);
    rl = static_cast<float>(d - r);
    q = static_cast<int>(k);
  }
  const float z = __fmul_rn(r, r), zl = fmaf(r, r, -z);
  // sin: r - r^3 / 6 + ...
  const float a = __fmul_rn(r, z), al = fmaf(r, zl, fmaf(r, z, -a));
  float w = __fmul_rn(a, -0.166666672f);
  float wl = fmaf(al, -0.166666672f, fmaf(a, 4.967054e-9f, fmaf(a, -0.166666672f, -w)));
  float tail = a * z * fmaf(z, fmaf(z, fmaf(z, -2.50521084e-8f, 2.75573192e-6f), -1.98412698e-4f), 8.33333333e-3f);
  float s = r + w;
  const float S = s + ((w - (s - r)) + (wl + tail + rl * fmaf(-0.5f, z, 1.f)));
  // cos: 1 - r^2 / 2 + r^4 / 24 - ...
  const float z2 = fmaf(2.f * r, rl, zl);
  const float b = __fmul_rn(z, z), bl = fmaf(2.f * z, z2, fmaf(z, z, -b));
  w = __fmul_rn(b, 0.0416666679f);
  wl = fmaf(bl, 0.0416666679f, fmaf(b, -1.2417635e-9f, fmaf(b, 0.0416666679f, -w)));
  tail = b * z * fmaf(z, fmaf(z, fmaf(z, 2.08767570e-9f, -2.75573192e-7f), 2.48015873e-5f), -1.38888889e-3f);
  s = fmaf(-0.5f, z, 1.f);
  const float c = s + w;
  const float C = c + ((w - (c - s)) + (fmaf(-0.5f, z, 1.f - s) + fmaf(-0.5f, z2, wl + tail)));
  sn = (q & 1) ? C : S;
  cs = (q & 1) ? S : C;
  if (q & 2) sn = -sn;
  if ((q + 1) & 2) cs = -cs;
}

// Two bf16 products, each rounded once to bf16 (the exact product of two
// bf16 values fits in fp32, so this equals rounding the fp32 product).
PA_DEVINL uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Position and cache slot of new token t from the varlen metadata, as
// pa_slot_mapping computes them (nano-vLLM learning note, prepare_prefill
// listing): request b owns tokens cu[b] .. cu[b+1]-1, at positions
// context_lens[b] - n_b + j; a padding row (length 0) and an inconsistent
// request get position 0 and slot -1.  With `report` the flags and the
// optional outputs are written.
PA_DEVINL void map_token_of(const NormRopeParams& p, int64_t t, int b, int s0, int s1, int L, bool report, int& pos,
                             int64_t& slot) {
  const int n = s1 - s0, start = L - n;
  pos = 0;
  slot = -1;
  unsigned int flag = 0;
  if (s0 < 0 || t < s0 || t >= s1 || static_cast<int64_t>(s1) > p.n_tokens) {
    flag = PA_DEVERR_BAD_LENGTH;  // cu_seqlens_q does not cover the token
  } else if (L == 0) {
    // a padding row: stored nowhere
  } else if (start < 0 || static_cast<int64_t>(L) > static_cast<int64_t>(p.maxp) * p.page_size) {
    flag = PA_DEVERR_BAD_LENGTH;
  } else {
    pos = start + static_cast<int>(t - s0);
    const int page = p.bt[static_cast<int64_t>(b) * p.maxp + (pos >> p.log2P)];
    if (page >= 0 && page < p.num_pages)
      slot = static_cast<int64_t>(page) * p.page_size + (pos & (p.page_size - 1));
    else
      flag = PA_DEVERR_BAD_PAGE;
  }
  if (report) {
    if (flag) raise_flag(p.err, flag);
    if (p.pos_out) p.pos_out[t] = pos;
    if (p.slots_out) p.slots_out[t] = slot;
  }
}

// The same for any batch: the token's request by binary search over cu.
PA_DEVINL void map_token(const NormRopeParams& p, int64_t t, bool report, int& pos, int64_t& slot) {
  int lo = 0, hi = p.batch - 1;  // the last request whose tokens start at or before t
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.cu[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  map_token_of(p, t, lo, p.cu[lo], p.cu[lo + 1], p.ctx[lo], report, pos, slot);
}

constexpr int kNrThreads = 128;
constexpr int kNrCtasPerSm = 8;
// 4-bit rows take more registers: 80 without recomputing values, so 5 CTAs
// (16384 tokens of 16 q- and 8 kv-heads: 63.9 us; 4 and 6 CTAs 68.4 and 66.1 us
// where 5 took 63.3).
constexpr int kNrCtasPerSmQ4 = 5;
constexpr int kNrMaxPerCta = 2048;

// Shared-memory bytes of one token's stage: its q, k and v rows.
__host__ __device__ constexpr int nr_stage_bytes(int hq, int hkv, int hd, int e) { return (hq + 2 * hkv) * hd * e; }

// A CTA walks the tokens t = blockIdx.x, blockIdx.x + gridDim.x, ...: one
// thread copies each token's q, k and v rows into a two-stage shared-memory
// ring with bulk async copies (TMA engine), two tokens ahead, so the rows of
// the next token stream in while the current one is normed and rotated.
// A group of LPH lanes handles one head: lane l owns elements [4l, 4l+4) of
// the first half and the same of the second half, so each lane holds both
// members of its rotation pairs.  Values are rounded to the storage type
// after the normalisation, after the weight and after the rotation (the
// casts of the Qwen3 norm and rotary in the nano-vLLM learning note); for
// bf16 the element arithmetic runs on fp32 pairs (packed multiplies and FMAs,
// one two-lane conversion per rounding).
//
// GS != 0: the cache holds 4-bit rows with groups of GS dims (q4_common.cuh).
// The rotated k (rounded to the storage type, as a cache of that type would
// hold it) goes back into the stage in place of the k it came from; the warp
// then takes eight consecutive dims a lane of these heads' k and v rows and
// quantises the two together, which shares the work on the groups' parameters
// (quantising k from the rotation's registers and v apart took 3240 instructions
// a token instead of 2900).  A code moves by a whole step when its value crosses
// a border by an ulp, so here the norm and the rotation are the plain formulas,
// operation by operation in fp32: squares rounded and added, products and sums of
// the rotation rounded each, sines and cosines rounded from more than fp32 (3189
// instructions a token: 16384 tokens 63.9 us; 3138 and 62.4 with angles of float pairs
// alone, 60.8 with the plain caches' arithmetic).  The order in which the squares
// are added (32 elements apart, then neighbours in pairs) is no more exact than
// another; it is the interface's, stated in its header, so that a row's codes can be
// worked out elsewhere bit for bit.  A lane's pairs lie so that it holds the elements
// that are added first.
template <typename T, int HD, int GS>
__global__ void __launch_bounds__(kNrThreads, GS ? kNrCtasPerSmQ4 : 0)
    norm_rope_kv_write_kernel(const NormRopeParams p) {
  constexpr int E = sizeof(T);
  constexpr int PE = 4;
  constexpr int LPH = HD / (2 * PE);  // lanes per head
  constexpr int HPW = 32 / LPH;       // heads per warp pass
  extern __shared__ __align__(128) unsigned char nr_smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / LPH, l = lane % LPH;
  const int row_q = p.hq * HD * E, row_kv = p.hkv * HD * E;
  const int stage_bytes = row_q + 2 * row_kv;
  unsigned char* stages = nr_smem;
  uint64_t* full = reinterpret_cast<uint64_t*>(nr_smem + 2 * stage_bytes);
  float* cs_s = reinterpret_cast<float*>(full + 2);   // [HD / 2]
  float* sn_s = cs_s + HD / 2;
  // the CTA's tokens' (position, slot) when they come from the metadata
  longlong2* meta_s = reinterpret_cast<longlong2*>(sn_s + HD / 2);
  __shared__ int abort_flag;
  pdl_trigger();  // as in kv_write_kernel: the prefill planner may start beside this grid

  const int64_t t0 = blockIdx.x, dt = gridDim.x;
  const int n_mine = static_cast<int>((p.n_tokens - t0 + dt - 1) / dt);  // tokens of this CTA
  auto issue = [&](int i) {  // thread 0: the copies of the CTA's i-th token into stage i & 1
    const int64_t t = t0 + i * dt;
    unsigned char* st = stages + (i & 1) * stage_bytes;
    mbar_arrive_expect_tx(&full[i & 1], static_cast<uint32_t>(stage_bytes));
    bulk_g2s(st, static_cast<const char*>(p.q) + t * p.q_stride * E, row_q, &full[i & 1]);
    bulk_g2s(st + row_q, static_cast<const char*>(p.k) + t * p.k_stride * E, row_kv, &full[i & 1]);
    bulk_g2s(st + row_q + row_kv, static_cast<const char*>(p.v) + t * p.v_stride * E, row_kv, &full[i & 1]);
  };
  if (threadIdx.x == 0) {
    mbar_init(&full[0], 1);
    mbar_init(&full[1], 1);
    abort_flag = 0;
    fence_mbar_init();
    if (n_mine > 0) issue(0);
    if (n_mine > 1) issue(1);
  }

  // The lane's rotation pairs i: elements i and HD / 2 + i of a head.
  constexpr bool kSplit = GS != 0 && HD == 128;  // i = 2l, 2l + 1, 32 + 2l, 33 + 2l; else 4l ... 4l + 3
  auto load_pairs = [&](const T* row, float (&x)[PE]) {
    if constexpr (kSplit) {
      load_two(row + 2 * l, x[0], x[1]);
      load_two(row + 32 + 2 * l, x[2], x[3]);
    } else {
      Vec4<T>::load(row + l * PE, x);
    }
  };
  // a + b where a or b is a product: an addition would be contracted with it, a
  // multiply-add by a 1 that the compiler does not know (theta^0) is not.
  [[maybe_unused]] const float2 one = make_float2(p.inv_freq_hi[0], p.inv_freq_hi[0]);
  [[maybe_unused]] auto plus = [&](float2 a, float2 b) { return ffma2(a, one, b); };
  float wq_a[PE], wq_b[PE], wk_a[PE], wk_b[PE];
  load_pairs(static_cast<const T*>(p.wq), wq_a);
  load_pairs(static_cast<const T*>(p.wq) + HD / 2, wq_b);
  load_pairs(static_cast<const T*>(p.wk), wk_a);
  load_pairs(static_cast<const T*>(p.wk) + HD / 2, wk_b);
  // bf16: the weights as bf16 pairs for the packed multiply
  uint32_t wq_a2[PE / 2], wq_b2[PE / 2], wk_a2[PE / 2], wk_b2[PE / 2];
#pragma unroll
  for (int e2 = 0; e2 < PE / 2; ++e2) {
    wq_a2[e2] = pack_bf16x2(wq_a[2 * e2], wq_a[2 * e2 + 1]);
    wq_b2[e2] = pack_bf16x2(wq_b[2 * e2], wq_b[2 * e2 + 1]);
    wk_a2[e2] = pack_bf16x2(wk_a[2 * e2], wk_a[2 * e2 + 1]);
    wk_b2[e2] = pack_bf16x2(wk_b[2 * e2], wk_b[2 * e2 + 1]);
  }
  // a token's position and slot: from the inputs, or mapped from the varlen
  // metadata for all of the CTA's tokens at once by warp 1 (the mapping's
  // dependent loads overlap the first token's copies)
  const bool mapped = p.positions == nullptr;
  if (mapped && warp == 1) {
    if (p.batch < 32) {
      // up to 31 requests: their cu and lengths in the lanes, one load each,
      // so a token's request is a count of lanes, not a chain of loads
      const int cu_l = lane <= p.batch ? p.cu[lane] : INT_MAX;
      const int ctx_l = lane < p.batch ? p.ctx[lane] : 0;
      for (int k0 = 0; k0 < n_mine; k0 += 32) {
        const int k = k0 + lane;
        const int64_t t = t0 + static_cast<int64_t>(k) * dt;
        int b = -1;
#pragma unroll 1
        for (int j = 0; j < p.batch; ++j) b += __shfl_sync(0xffffffffu, cu_l, j) <= t;
        b = max(b, 0);
        const int s0 = __shfl_sync(0xffffffffu, cu_l, b), s1 = __shfl_sync(0xffffffffu, cu_l, b + 1);
        const int L = __shfl_sync(0xffffffffu, ctx_l, b);
        if (k < n_mine) {
          int pos;
          int64_t slot;
          map_token_of(p, t, b, s0, s1, L, true, pos, slot);
          meta_s[k] = make_longlong2(pos, slot);
        }
      }
    } else {
      for (int k = lane; k < n_mine; k += 32) {
        int pos;
        int64_t slot;
        map_token(p, t0 + k * dt, true, pos, slot);
        meta_s[k] = make_longlong2(pos, slot);
      }
    }
  }
  auto token_meta = [&](int i, int& pos, int64_t& slot) {
    if (mapped) {
      const longlong2 m = meta_s[i];
      pos = static_cast<int>(m.x);
      slot = m.y;
    } else {
      pos = p.positions[t0 + i * dt];
      slot = p.slots[t0 + i * dt];
    }
  };
  cta_sync();
  int pos_next = 0;
  int64_t slot_next = -1;
  if (n_mine > 0) token_meta(0, pos_next, slot_next);

  int done = 0;  // tokens finished (their stages consumed)
  for (int i = 0; i < n_mine; ++i) {
    const int64_t t = t0 + i * dt;
    const int pos = pos_next;
    const int64_t slot = slot_next;
    if (i + 1 < n_mine) token_meta(i + 1, pos_next, slot_next);  // the next token's, one token ahead
    const bool slot_ok = slot >= 0 && slot < p.num_slots;
    if (!slot_ok && slot != -1 && threadIdx.x == 0) raise_flag(p.err, PA_DEVERR_BAD_SLOT);
    // cos / sin of the token's HD/2 pair indices, one thread per pair, of the
    // angle pos * theta^(-2i/HD) formed in two-float arithmetic: reduced modulo
    // 2*pi and evaluated by the special-function unit, or (4-bit rows) reduced
    // modulo pi/2 and evaluated by sincos_pair's series
    if (threadIdx.x < HD / 2) {
      float sv, cv;
      if constexpr (GS == 0) {
        const float r = reduce_angle(pos, p.inv_freq_hi[threadIdx.x], p.inv_freq_lo[threadIdx.x]);
        __sincosf(r, &sv, &cv);
      } else {
        sincos_pair(pos, p.inv_freq_hi[threadIdx.x], p.inv_freq_lo[threadIdx.x], p.inv_freq[threadIdx.x], sv, cv);
      }
      cs_s[threadIdx.x] = cv;
      sn_s[threadIdx.x] = sv;
    }
    const bool ok = mbar_wait_bounded(&full[i & 1], (i >> 1) & 1, &abort_flag, p.err);
    if (!__syncthreads_and(ok)) break;  // cos / sin written, every thread past its wait
    float cs[PE], sn[PE], nsn[PE];
#pragma unroll
    for (int e = 0; e < PE; ++e) {
      const int i = kSplit ? e / 2 * 32 + 2 * l + e % 2 : l * PE + e;
      cs[e] = cs_s[i];
      sn[e] = sn_s[i];
      nsn[e] = -sn[e];
    }
    unsigned char* st = stages + (i & 1) * stage_bytes;
    [[maybe_unused]] const uint32_t q4_codes = static_cast<uint32_t>(p.hkv) * (HD / 2),
                                    q4_pars = static_cast<uint32_t>(p.q4_row_bytes) - q4_codes,
                                    q4_t = static_cast<uint32_t>(slot);
    const int nheads = p.hq + p.hkv;
    for (int hh = warp * HPW + sub; hh - sub < nheads; hh += (kNrThreads / 32) * HPW) {
      const bool active = hh < nheads;
      const bool isq = hh < p.hq;
      const T* src = reinterpret_cast<const T*>(st) + static_cast<int64_t>(active ? hh : 0) * HD;
      float xa[PE] = {0.f, 0.f, 0.f, 0.f}, xb[PE] = {0.f, 0.f, 0.f, 0.f};
      if (active) {
        load_pairs(src, xa);
        load_pairs(src + HD / 2, xb);
      }
      float ss;
      if constexpr (GS == 0) {
        float2 ss2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < PE; e += 2) {
          ss2 = ffma2(make_float2(xa[e], xa[e + 1]), make_float2(xa[e], xa[e + 1]), ss2);
          ss2 = ffma2(make_float2(xb[e], xb[e + 1]), make_float2(xb[e], xb[e + 1]), ss2);
        }
        ss = ss2.x + ss2.y;
#pragma unroll
        for (int m = LPH / 2; m >= 1; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
      } else {
        // t + x^2, the square rounded (a bf16's is exact)
        auto add_square = [&](float2 t, float x, float y) {
          const float2 v = make_float2(x, y);
          return sizeof(T) == 2 ? ffma2(v, v, t) : plus(fmul2(v, v), t);
        };
        const float2 zero = make_float2(0.f, 0.f);
        float2 t0 = add_square(zero, xa[0], xa[1]);
        if constexpr (HD == 128) {  // elements j, j + 32, j + 64, j + 96
          t0 = add_square(add_square(add_square(t0, xa[2], xa[3]), xb[0], xb[1]), xb[2], xb[3]);
          ss = t0.x + t0.y;
        } else {                    // j, j + 32
          t0 = add_square(t0, xb[0], xb[1]);
          const float2 t1 = add_square(add_square(zero, xa[2], xa[3]), xb[2], xb[3]);
          ss = (t0.x + t0.y) + (t1.x + t1.y);
        }
#pragma unroll
        for (int m = 1; m < LPH; m <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
      }
      // a 4-bit group's reduction takes the whole warp, heads past the last included
      if constexpr (GS == 0) {
        if (!active) continue;
      }
      const float r = rsqrtf(ss * (1.0f / HD) + p.eps);
      T* dst = isq ? static_cast<T*>(p.q_out) + (t * p.hq + hh) * HD
                   : GS == 0 ? static_cast<T*>(p.k_cache) + (slot * p.hkv + (hh - p.hq)) * HD : const_cast<T*>(src);
      const bool store = GS == 0 ? isq || slot_ok : active;  // (4-bit: k into the stage)
      if constexpr (sizeof(T) == 2) {
        // y_a = n_a cos - n_b sin, y_b = n_b cos + n_a sin on fp32 pairs
        uint32_t wa[PE / 2], wb[PE / 2];
        const float2 r2 = make_float2(r, r);
#pragma unroll
        for (int e2 = 0; e2 < PE / 2; ++e2) {
          const int e = 2 * e2;
          const float2 ta = fmul2(make_float2(xa[e], xa[e + 1]), r2);
          const float2 tb = fmul2(make_float2(xb[e], xb[e + 1]), r2);
          const float2 na = bf16x2_to_float2(mul_bf16x2(pack_bf16x2(ta.x, ta.y), isq ? wq_a2[e2] : wk_a2[e2]));
          const float2 nb = bf16x2_to_float2(mul_bf16x2(pack_bf16x2(tb.x, tb.y), isq ? wq_b2[e2] : wk_b2[e2]));
          const float2 c2 = make_float2(cs[e], cs[e + 1]);
          const float2 s2 = make_float2(sn[e], sn[e + 1]), ns2 = make_float2(nsn[e], nsn[e + 1]);
          const float2 ya = GS == 0 ? ffma2(nb, ns2, fmul2(na, c2)) : plus(fmul2(na, c2), fmul2(nb, ns2));
          const float2 yb = GS == 0 ? ffma2(nb, c2, fmul2(na, s2)) : plus(fmul2(nb, c2), fmul2(na, s2));
          wa[e2] = pack_bf16x2(ya.x, ya.y);
          wb[e2] = pack_bf16x2(yb.x, yb.y);
        }
        if (store) {
          if constexpr (kSplit) {
#pragma unroll
            for (int e2 = 0; e2 < PE / 2; ++e2) {
              *reinterpret_cast<uint32_t*>(dst + e2 * 32 + 2 * l) = wa[e2];
              *reinterpret_cast<uint32_t*>(dst + HD / 2 + e2 * 32 + 2 * l) = wb[e2];
            }
          } else {
            *reinterpret_cast<uint2*>(dst + l * PE) = make_uint2(wa[0], wa[1]);
            *reinterpret_cast<uint2*>(dst + HD / 2 + l * PE) = make_uint2(wb[0], wb[1]);
          }
        }
      } else {
        float ya[PE], yb[PE];
#pragma unroll
        for (int e = 0; e < PE; ++e) {
          const float na = round_to<T>(round_to<T>(xa[e] * r) * (isq ? wq_a[e] : wk_a[e]));
          const float nb = round_to<T>(round_to<T>(xb[e] * r) * (isq ? wq_b[e] : wk_b[e]));
          ya[e] = GS == 0 ? round_to<T>(na * cs[e] - nb * sn[e])
                          : round_to<T>(__fmul_rn(na, cs[e]) + __fmul_rn(nb, nsn[e]));
          yb[e] = GS == 0 ? round_to<T>(nb * cs[e] + na * sn[e])
                          : round_to<T>(__fmul_rn(nb, cs[e]) + __fmul_rn(na, sn[e]));
        }
        if (store) {
          if constexpr (kSplit) {
#pragma unroll
            for (int e = 0; e < PE; e += 2) {
              *reinterpret_cast<float2*>(dst + e * 16 + 2 * l) = make_float2(ya[e], ya[e + 1]);
              *reinterpret_cast<float2*>(dst + HD / 2 + e * 16 + 2 * l) = make_float2(yb[e], yb[e + 1]);
            }
          } else {
            Vec4<T>::store(dst + l * PE, ya);
            Vec4<T>::store(dst + HD / 2 + l * PE, yb);
          }
        }
      }
      if constexpr (GS != 0) {
        if (hh - sub + HPW > p.hq) {  // the pass holds a k head (the same for the whole warp)
          __syncwarp();               // its rotated k is in the stage
          const int h = hh - p.hq;
          const bool mine = active && !isq;
          uint32_t kw[kQ4Words<T>] = {}, vw[kQ4Words<T>] = {};
          if (mine) {
#pragma unroll
            for (int e = 0; e < kQ4Words<T>; e += 4) {
              const uint4 a = *reinterpret_cast<const uint4*>(st + row_q + (h * HD + l * 8) * E + e * 4);
              const uint4 b = *reinterpret_cast<const uint4*>(st + row_q + row_kv + (h * HD + l * 8) * E + e * 4);
              kw[e] = a.x; kw[e + 1] = a.y; kw[e + 2] = a.z; kw[e + 3] = a.w;
              vw[e] = b.x; vw[e + 1] = b.y; vw[e + 2] = b.z; vw[e + 3] = b.w;
            }
          }
          uint32_t kc, vc, kp, vp;
          q4_quantise8_pair<T>(kw, vw, GS / 8, kc, vc, kp, vp);
          if (mine && slot_ok) {
            char* kr = static_cast<char*>(p.k_cache) + slot * p.q4_row_bytes;
            char* vr = static_cast<char*>(p.v_cache) + slot * p.q4_row_bytes;
            const uint32_t co = q4_swz((h * (HD / 8) + l) * 4, q4_codes, q4_t);
            *reinterpret_cast<uint32_t*>(kr + co) = kc;
            *reinterpret_cast<uint32_t*>(vr + co) = vc;
            if (l % (GS / 8) == 0) {
              const uint32_t po = q4_codes + q4_swz((h * (HD / GS) + l / (GS / 8)) * 4, q4_pars, q4_t);
              *reinterpret_cast<uint32_t*>(kr + po) = kp;
              *reinterpret_cast<uint32_t*>(vr + po) = vp;
            }
          }
          // the rotated k's stores come before the copies that refill the stage
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
      }
    }
    if constexpr (GS != 0) {
      // (the v row is written with its k heads)
    } else if (slot_ok) {  // the v row, unchanged, into its slot
      const unsigned char* vsrc = st + row_q + row_kv;
      char* vdst = static_cast<char*>(p.v_cache) + slot * row_kv;
      for (int ch = threadIdx.x; ch < row_kv / 16; ch += kNrThreads)
        stg16(vdst + ch * 16, *reinterpret_cast<const uint4*>(vsrc + ch * 16));
    }
    cta_sync();  // every thread is done with the stage and with cos / sin
    if (threadIdx.x == 0 && i + 2 < n_mine) issue(i + 2);
    done = i + 1;
  }
  if (threadIdx.x == 0) {
    // after an abort, copies issued for tokens not reached may still land:
    // wait for them (time only) before the CTA exits
    for (int i = done; i < n_mine && i < done + 2; ++i) {
      const uint64_t tw = global_timer_ns();
      while (!mbar_try_wait(&full[i & 1], (i >> 1) & 1) && global_timer_ns() - tw < kWaitLimitNs) {
      }
    }
  }
}

// The kernel for rows of the storage type (gs = 0) or 4-bit rows with groups of gs dims.
template <typename T, int HD>
const void* norm_rope_fn(int gs) {
  if (gs == 0) return reinterpret_cast<const void*>(norm_rope_kv_write_kernel<T, HD, 0>);
  if constexpr (HD == 128)
    if (gs == 128) return reinterpret_cast<const void*>(norm_rope_kv_write_kernel<T, HD, 128>);
  return gs == 64 ? reinterpret_cast<const void*>(norm_rope_kv_write_kernel<T, HD, 64>)
                  : reinterpret_cast<const void*>(norm_rope_kv_write_kernel<T, HD, 32>);
}

}  // namespace

cudaError_t launch_slot_mapping(const SlotMapParams& p, cudaStream_t s) {
  if (p.batch == 0) return cudaSuccess;
  slot_mapping_kernel<<<p.batch, 128, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_kv_write(const KvWriteParams& p, cudaStream_t s) {
  if (p.n_tokens == 0) return cudaSuccess;
  DeviceInfo di;
  cudaError_t e = current_device_info(&di);
  if (e != cudaSuccess) return e;
  const int64_t total = p.n_tokens * (p.row_bytes / 16);
  const int64_t blocks = std::min<int64_t>((total + 255) / 256, static_cast<int64_t>(di.sm_count) * 8);
  kv_write_kernel<<<static_cast<unsigned>(blocks), 256, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_norm_rope_kv_write(int dtype, int head_dim, const NormRopeParams& p, cudaStream_t s) {
  if (p.n_tokens == 0) return cudaSuccess;
  DeviceInfo di;
  cudaError_t e = current_device_info(&di);
  if (e != cudaSuccess) return e;
  const int es = dtype == PA_BF16 ? 2 : 4;
  // one wave of CTAs walking the tokens, with at most kNrMaxPerCta tokens
  // each (the mapped tokens' positions and slots are kept in shared memory)
  const int64_t wave = static_cast<int64_t>(di.sm_count) * (p.q4_group_size ? kNrCtasPerSmQ4 : kNrCtasPerSm);
  const unsigned grid = static_cast<unsigned>(
      std::max(std::min<int64_t>(p.n_tokens, wave), (p.n_tokens + kNrMaxPerCta - 1) / kNrMaxPerCta));
  const int64_t per_cta = (p.n_tokens + grid - 1) / grid;  // tokens of the busiest CTA
  const size_t smem = 2 * static_cast<size_t>(nr_stage_bytes(p.hq, p.hkv, head_dim, es)) + 2 * sizeof(uint64_t) +
                      head_dim * sizeof(float) + (p.positions == nullptr ? per_cta * sizeof(longlong2) : 0);
  if (smem > static_cast<size_t>(di.max_smem_optin)) return cudaErrorInvalidValue;
  const int gs = p.q4_group_size;
  const void* fn = dtype == PA_BF16
                       ? (head_dim == 128 ? norm_rope_fn<__nv_bfloat16, 128>(gs) : norm_rope_fn<__nv_bfloat16, 64>(gs))
                       : (head_dim == 128 ? norm_rope_fn<float, 128>(gs) : norm_rope_fn<float, 64>(gs));
  if (smem > 48 * 1024) {
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  void* args[] = {const_cast<NormRopeParams*>(&p)};
  e = cudaLaunchKernel(fn, dim3(grid), dim3(kNrThreads), args, smem, s);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace pa
