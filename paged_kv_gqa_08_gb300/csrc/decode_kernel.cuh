// The kernel of batched GQA decode attention over a paged KV cache (sm_103a):
// instantiated over all of a request's keys in decode.cu, and over keys with a
// range left out (kRange: a sliding window with sinks, or the tokens after a
// prefix that other requests share) in decode_range.cu.
//
// Semantics (nano-vLLM learning note, Attention.forward and prepare_decode
// listings): each request's single query attends to all context_lens[b] keys
// of its block table, after this step's KV write.
//
// Design (HBM-bound):
//   * The keys of all requests are cut into chunks of T tokens (T divides the
//     page size, so a chunk lies inside one page and is one contiguous run of
//     T * Hkv * head_dim elements).  The global chunk list is split evenly
//     over the CTAs of one wave ("plan" kernel), so every SM streams the same
//     number of bytes whatever the length mix.  A request cut across CTAs
//     gets per-CTA (o, log2-sum-exp) partials, merged by a second kernel
//     (split-KV / flash-decoding).  The cut depends only on context_lens, so
//     results are bitwise independent of physical page ids.
//   * One producer warp issues 1-D bulk async copies (TMA engine) of each
//     chunk's K and V rows into a 3-stage shared-memory ring, with mbarrier
//     completion and an evict-first L2 hint.  Its 32 lanes look up block-table
//     entries for 32 chunks at a time.
//   * One consumer warp per kv-head reads its head's rows of the chunk, so
//     one K/V byte feeds all G q-heads of the group.  Two consumers:
//     - CUDA cores (fp32, or head_dim 64): each lane owns 16
//       bytes of a row; dot products use packed fp32x2 FMA, partial sums are
//       reduced with a halving butterfly of warp shuffles, the online
//       softmax runs in base 2 with the scale folded into q.
//     - tensor cores (bf16, head_dim 128, any group of up to 8): per 16-token
//       chunk, S = Q K^T and O += P V as mma.sync m16n8k16 with the group's
//       q-heads as the (zero-padded) 16 rows; K and V fragments come by
//       ldmatrix from stage rows padded by 16 bytes (each row its own copy),
//       so the loads are free of bank conflicts.  Far fewer instructions per
//       byte: the CUDA-core consumer is issue-bound from G = 4 on.
//   * Every wait is bounded (pa::mbar_wait_bounded): a kernel never hangs.
#pragma once

#include "decode_shared.cuh"

namespace pa {
namespace {

constexpr int kTPL = 4;          // tokens per lane per chunk
constexpr int kStages = 3;       // shared-memory ring depth (CUDA-core consumers, up to two CTAs per SM)
constexpr int kStagesMma = 3;    // ring depth of the tensor-core consumers (one CTA per SM)
constexpr int kMmaTok = 16;      // tokens per chunk of the tensor-core consumers

__host__ __device__ constexpr int ilog2c(int x) { return x <= 1 ? 0 : 1 + ilog2c(x / 2); }
__host__ __device__ constexpr int pow2ceil(int x) { return x <= 1 ? 1 : 2 * pow2ceil((x + 1) / 2); }

template <typename T, int HD>
struct Geom {
  static constexpr int E = sizeof(T);
  static constexpr int DPL = 16 / E;      // elements a lane holds of one row
  static constexpr int NPR = DPL / 2;     // float2 pairs per lane
  static constexpr int LPR = HD / DPL;    // lanes covering one head row
  static constexpr int RPI = 32 / LPR;    // rows one warp instruction covers
  static constexpr int TOK = kTPL * RPI;  // tokens per chunk
  static constexpr int RB = HD * E;       // bytes of one head row
};

// ---------------------------------------------------------------------------
// halving butterfly: reduce CUR values over the lanes of a row group, keeping
// half of the (partially summed) values per step.
// ---------------------------------------------------------------------------
template <int CUR, int M>
struct Butterfly {
  template <int N>
  static PA_DEVINL void run(float (&a)[N], int lane) {
    if constexpr (CUR >= 2) {
      constexpr int H = CUR / 2;
      const bool upper = (lane & M) != 0;
#pragma unroll
      for (int u = 0; u < H; ++u) {
        const float send = upper ? a[u] : a[u + H];
        const float keep = upper ? a[u + H] : a[u];
        a[u] = keep + __shfl_xor_sync(0xffffffffu, send, M);
      }
      if constexpr (M > 1) Butterfly<H, M / 2>::run(a, lane);
    } else {
      a[0] += __shfl_xor_sync(0xffffffffu, a[0], M);
      if constexpr (M > 1) Butterfly<1, M / 2>::run(a, lane);
    }
  }
};

// The halving levels of Butterfly alone (CUR values -> 1 over lane bits M,
// M/2, ...), for reducing a sub-array whose levels come first.
template <int CUR, int M>
struct Halve {
  template <int N>
  static PA_DEVINL void run(float (&a)[N], int lane) {
    if constexpr (CUR >= 2) {
      static_assert(M >= 1, "one lane bit per halving level");
      constexpr int H = CUR / 2;
      const bool upper = (lane & M) != 0;
#pragma unroll
      for (int u = 0; u < H; ++u) {
        const float send = upper ? a[u] : a[u + H];
        const float keep = upper ? a[u + H] : a[u];
        a[u] = keep + __shfl_xor_sync(0xffffffffu, send, M);
      }
      Halve<H, M / 2>::run(a, lane);
    }
  }
};

// Floats per token row of the probability tile: each probability is stored
// twice, (p, p), so that the PV products read ready-made fp32 pairs, and the
// row is padded to whole 16-byte vectors.
__host__ __device__ constexpr int p_row_floats(int G) { return 2 * (G <= 2 ? 2 : G <= 4 ? 4 : 8); }

template <typename T, int NPR>
PA_DEVINL void unpack16(const uint4 w, float2 (&f)[NPR]) {
  if constexpr (sizeof(T) == 2) {
    f[0] = bf16x2_to_float2(w.x);
    f[1] = bf16x2_to_float2(w.y);
    f[2] = bf16x2_to_float2(w.z);
    f[3] = bf16x2_to_float2(w.w);
  } else {
    f[0] = make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
    f[1] = make_float2(__uint_as_float(w.z), __uint_as_float(w.w));
  }
}

template <typename T, int NPR>
PA_DEVINL uint4 pack16(const float2 (&f)[NPR], float s) {
  uint4 w;
  if constexpr (sizeof(T) == 2) {
    w.x = pack_bf16x2(f[0].x * s, f[0].y * s);
    w.y = pack_bf16x2(f[1].x * s, f[1].y * s);
    w.z = pack_bf16x2(f[2].x * s, f[2].y * s);
    w.w = pack_bf16x2(f[3].x * s, f[3].y * s);
  } else {
    w.x = __float_as_uint(f[0].x * s);
    w.y = __float_as_uint(f[0].y * s);
    w.z = __float_as_uint(f[1].x * s);
    w.w = __float_as_uint(f[1].y * s);
  }
  return w;
}

// ---------------------------------------------------------------------------
// tensor-core consumer (bf16, head_dim 128, up to 8 q-heads per kv-head)
// ---------------------------------------------------------------------------
// mma.sync fragments (PTX ISA, m16n8k16 with .row.col): lane l is
// in row group gq = l / 4 and thread-in-group tq = l % 4.  A holds rows gq and
// gq + 8; B holds column gq; C holds rows gq (c0, c1) and gq + 8 (c2, c3) at
// columns 2 tq, 2 tq + 1.  Here the rows are the group's q-heads (G <= 8 of
// them, padded to 16 with zero rows), so only c0 / c1 of lanes with gq < G
// carry results.
PA_DEVINL void mma_16816(float (&d)[2], uint32_t a0, uint32_t a2, uint32_t b0, uint32_t b1) {
  [[maybe_unused]] float x2, x3;  // rows gq + 8 (padding), discarded
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %10, %10};"
      : "+f"(d[0]), "+f"(d[1]), "=f"(x2), "=f"(x3)
      : "r"(a0), "r"(0u), "r"(a2), "r"(0u), "r"(b0), "r"(b1), "f"(0.f));
}

// Four 8x8 b16 matrices from shared memory; lanes 8i .. 8i+7 give the row
// addresses of matrix i.  .trans delivers each matrix transposed.
PA_DEVINL void ldsm_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

PA_DEVINL void ldsm_x4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

// The consumer warp of kv-head `warp` for the chunks [x0, x1) of CTA c: per
// 16-token chunk, S = Q K^T as 16 m16n8k16 MMAs in two chains (K^T fragments
// by ldmatrix from the padded stage rows), the online softmax in base 2 on
// the S fragments, and O += P V as 16 m16n8k16 MMAs (P straight from the S
// fragments, V fragments by transposed ldmatrix).  Same results contract as the CUDA-core
// consumer: whole requests to `out`, shares to the partial slots.
template <int G, int NS, bool kRange>
PA_DEVINL void mma_consumer(const KParams& p, unsigned char* smem, uint64_t* full, uint64_t* empty, const int4* meta,
                            volatile int* abort_flag, int x0, int x1, int c) {
  constexpr int RB = 256;  // bytes of one head row (128 bf16)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = warp;
  const int gq = lane >> 2, tq = lane & 3;
  const bool row_live = gq < G;
  const int lrow = lane & 7, lmat = lane >> 3;  // ldmatrix: this lane's row and matrix
  const uint32_t smem0 = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
  uint32_t qa[8][2];  // A fragments of q for k-steps of 16 dims: dims 2tq.. and 2tq+8.. of row gq
  float o[16][2];     // O row gq, columns 8j + 2tq, 8j + 2tq + 1
  float m_run = -INFINITY, l_part = 0.f;
  int b = 0;
  uint4 nrow = make_uint4(0, 0, 0, 0);  // this head's piece of the request's new K (lanes 0-15) / V row

  for (int x = x0, it = 0; x < x1; ++x, ++it) {
    const int s = it % NS;
    if (!mbar_wait_bounded(&full[s], (it / NS) & 1, abort_flag, p.err)) break;
    const int4 md = meta[s];
    b = md.x;
    const int n = md.y, flags = md.z;

    if (flags & 1) {  // first chunk of this CTA's share of request b
      if ((flags & 16) && p.k_new != nullptr)  // the share ends the request: its new row, early
        nrow = *reinterpret_cast<const uint4*>(
            (lane < 16 ? p.k_new + static_cast<int64_t>(b) * p.k_new_stride
                       : p.v_new + static_cast<int64_t>(b) * p.v_new_stride) + h * RB + (lane & 15) * 16);
      const char* qrow = p.q + (static_cast<int64_t>(b) * p.Hq + h * G + (row_live ? gq : 0)) * RB;
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        qa[ks][0] = row_live ? *reinterpret_cast<const uint32_t*>(qrow + (ks * 16 + 2 * tq) * 2) : 0u;
        qa[ks][1] = row_live ? *reinterpret_cast<const uint32_t*>(qrow + (ks * 16 + 8 + 2 * tq) * 2) : 0u;
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) o[j][0] = o[j][1] = 0.f;
      m_run = -INFINITY;
      l_part = 0.f;
    }

    unsigned char* kst = smem + static_cast<size_t>(s) * 2 * p.chunk_bytes + h * RB;
    unsigned char* vst = kst + p.chunk_bytes;
    if (md.w >= 0) {
      // fused KV write: this head's piece of the new row (row n - 1), read by
      // the consumer from k_new / v_new at the start of the share (not copied
      // by the producer, so they may be in pinned host memory), goes into the
      // stage for the products and to its slot
      const int64_t dst_off = static_cast<int64_t>(md.w) * p.row_bytes + h * RB;
      *reinterpret_cast<uint4*>((lane < 16 ? kst : vst) + (n - 1) * p.row_pitch + (lane & 15) * 16) = nrow;
      char* dst = const_cast<char*>(lane < 16 ? p.k_cache : p.v_cache) + dst_off + (lane & 15) * 16;
      stg16(dst, nrow);
    }
    if (n < kMmaTok) {
      // a ragged chunk: the V rows past its end meet probability 0 and must be
      // finite (they may hold another chunk's data or nothing yet)
      for (int r = n; r < kMmaTok; ++r)
        if (lane < 16) *reinterpret_cast<uint4*>(vst + r * p.row_pitch + lane * 16) = make_uint4(0, 0, 0, 0);
    }
    // rows [hole_a, hole_z) of the chunk are left out: not copied, probability 0
    const int hole_a = kRange ? (flags >> 8) & 31 : 0, hole_z = kRange ? (flags >> 16) & 31 : 0;
    if constexpr (kRange) {
      for (int r = hole_a; r < hole_z; ++r)
        if (lane < 16) *reinterpret_cast<uint4*>(vst + r * p.row_pitch + lane * 16) = make_uint4(0, 0, 0, 0);
    }
    if (md.w >= 0 || n < kMmaTok || (kRange && hole_z > hole_a)) {
      // the fence orders these stores before the copies that refill the stage later
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
    }

    // S = Q K^T for the chunk's tokens 0-7 (s0) and 8-15 (s1): row gq, tokens
    // 2tq, 2tq + 1 (+ 8); two independent accumulator chains
    const uint32_t ka = smem0 + static_cast<uint32_t>(kst - smem) + lrow * p.row_pitch + lmat * 16;
    const uint32_t ka8 = ka + 8 * p.row_pitch;
    float s0[2] = {0.f, 0.f}, s1[2] = {0.f, 0.f};
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      uint32_t bf[4], bg[4];
      ldsm_x4(bf, ka + kk * 64);
      ldsm_x4(bg, ka8 + kk * 64);
      mma_16816(s0, qa[2 * kk][0], qa[2 * kk][1], bf[0], bf[1]);
      mma_16816(s1, qa[2 * kk][0], qa[2 * kk][1], bg[0], bg[1]);
      mma_16816(s0, qa[2 * kk + 1][0], qa[2 * kk + 1][1], bf[2], bf[3]);
      mma_16816(s1, qa[2 * kk + 1][0], qa[2 * kk + 1][1], bg[2], bg[3]);
    }
    const int tk = 2 * tq;
    auto seen = [&](int t) { return kRange ? t < n && (t < hole_a || t >= hole_z) : t < n; };
    const float v0 = seen(tk) ? s0[0] * p.scale_log2 : -INFINITY;
    const float v1 = seen(tk + 1) ? s0[1] * p.scale_log2 : -INFINITY;
    const float v2 = seen(tk + 8) ? s1[0] * p.scale_log2 : -INFINITY;
    const float v3 = seen(tk + 9) ? s1[1] * p.scale_log2 : -INFINITY;
    float mx = fmaxf(fmaxf(v0, v1), fmaxf(v2, v3));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    const float m_new = fmaxf(m_run, mx);
    const float m_use = m_new == -INFINITY ? 0.f : m_new;
    const float alpha = ex2_approx(m_run - m_use);
    const float p0 = ex2_approx(v0 - m_use), p1 = ex2_approx(v1 - m_use);
    const float p2 = ex2_approx(v2 - m_use), p3 = ex2_approx(v3 - m_use);
    l_part = l_part * alpha + ((p0 + p1) + (p2 + p3));
    if (__any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        o[j][0] *= alpha;
        o[j][1] *= alpha;
      }
    }
    m_run = m_new;

    // O += P V (m16n8k16: k = the chunk's 16 tokens); matrices of the
    // transposed loads: tokens 0-7 / 8-15 x dims d .. d+7 / d+8 .. d+15
    const uint32_t pa0 = pack_bf16x2(p0, p1), pa2 = pack_bf16x2(p2, p3);
    const uint32_t va = smem0 + static_cast<uint32_t>(vst - smem) + (lrow + (lmat & 1) * 8) * p.row_pitch +
                        (lmat >> 1) * 16;
#pragma unroll
    for (int nn = 0; nn < 8; ++nn) {
      uint32_t bf[4];
      ldsm_x4_t(bf, va + nn * 32);
      mma_16816(o[2 * nn], pa0, pa2, bf[0], bf[1]);
      mma_16816(o[2 * nn + 1], pa0, pa2, bf[2], bf[3]);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[s]);

    if (flags & 2) {  // last chunk of the share: write the result
      float l = l_part + __shfl_xor_sync(0xffffffffu, l_part, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      if (row_live) {
        const float inv = l > 0.f ? 1.f / l : 0.f;
        const int hq = h * G + gq;
        if (flags & 4) {
          char* dst = p.out + (static_cast<int64_t>(b) * p.Hq + hq) * RB + tq * 4;
#pragma unroll
          for (int j = 0; j < 16; ++j)
            *reinterpret_cast<uint32_t*>(dst + j * 16) = pack_bf16x2(o[j][0] * inv, o[j][1] * inv);
        } else {
          const int64_t slot = static_cast<int64_t>(c) + b;
          float* dst = p.o_part + (slot * p.Hq + hq) * 128 + 2 * tq;
#pragma unroll
          for (int j = 0; j < 16; ++j) *reinterpret_cast<float2*>(dst + 8 * j) = make_float2(o[j][0] * inv, o[j][1] * inv);
          // (kRange: a sum that is no number stays one for the merge)
          if (tq == 0) p.lse_part[slot * p.Hq + hq] = (kRange ? l != 0.f : l > 0.f) ? m_run + log2f(l) : -INFINITY;
        }
      }
      __syncwarp();
    }
  }
}

// ---------------------------------------------------------------------------
// the split-KV decode kernel
// ---------------------------------------------------------------------------
// The bf16 head_dim-128 kernels run their products on the tensor cores (see
// the MMA consumer below); fp32 and head_dim 64 on the CUDA cores.
template <typename T, int HD, int G>
constexpr bool kUseMma = std::is_same<T, __nv_bfloat16>::value && HD == 128;

template <typename T, int HD, int G, bool kRange>
// Register cap: a 9-warp CTA is charged as 10 warps, so two CTAs per SM need
// at most 96 registers per thread (CUDA-core consumers, G <= 4); larger groups
// and the tensor-core consumers run one CTA per SM with a deeper ring.
__global__ void __launch_bounds__(9 * 32) __maxnreg__((G <= 4 && !kUseMma<T, HD, G>) ? 96 : 168)
    decode_kernel(const KParams p) {
  constexpr bool kMma = kUseMma<T, HD, G>;
  constexpr int kStages = kMma ? kStagesMma : ::pa::kStages;
  using Gm = Geom<T, HD>;
  constexpr int LPR = Gm::LPR, RPI = Gm::RPI, NPR = Gm::NPR;
  constexpr int V = G * kTPL;
  constexpr int VP = pow2ceil(V);
  constexpr int VF = VP >= LPR ? VP / LPR : 1;          // values a lane keeps
  constexpr int DUP = VP >= LPR ? 0 : ilog2c(LPR / VP);  // low lane bits holding copies
  constexpr int IBITS = ilog2c(kTPL / VF);               // lane bits carrying the token index
  constexpr int GP = VP / kTPL;                          // heads padded to a power of two
  constexpr int PR = p_row_floats(G);
  static_assert(VF <= kTPL, "a lane's values must share one head");
  static_assert(GP <= LPR, "the head levels of the reduction fit in a row's lanes");

  extern __shared__ __align__(128) unsigned char smem[];
  const int c = blockIdx.x;
  const int NW = p.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  const int32_t* cs;  // [B+1] chunk prefix sums (of the CTA's own request: [2])
  const int cs0 = kRange && p.per_request ? c : 0;  // the request that they start with
  if (kRange && p.per_request) {
    int32_t* cs_s = reinterpret_cast<int32_t*>(smem + p.off_cs);
    const int cap = static_cast<int>(min(static_cast<int64_t>(p.max_ctx), static_cast<int64_t>(p.maxp) << p.log2P));
    bool bad;
    const int n = chunks_of<kRange>(p, c, cap, &bad);
    if (threadIdx.x == 0) {
      if (bad) raise_flag(p.err, PA_DEVERR_BAD_LENGTH);
      if (n == 0 && p.k_new != nullptr && p.slot_out) p.slot_out[c] = -1;
      cs_s[0] = 0;
      cs_s[1] = n;
    }
    if (n == 0) return;
    cta_sync();
    cs = cs_s;
  } else if (p.inline_plan) {
    int32_t* cs_s = reinterpret_cast<int32_t*>(smem + p.off_cs);
    plan_in_cta<kRange>(p, cs_s, cs_s + kInlinePlanMax + 1, c == 0);
    cs = cs_s;
  } else {
    pdl_wait();  // the plan kernel's chunk sums and CTA starts are complete
    cs = p.cs;
  }
  pdl_trigger();  // the merge kernel may start launching; it waits for this grid
  const bool alone = kRange && p.per_request;
  const int NC = cs[alone ? 1 : p.B];
  const int n_ctas = alone ? 1 : sharing_ctas<kRange>(p, NC), share = alone ? 0 : kRange ? min(c, n_ctas) : c;
  const int x0 = static_cast<int>((static_cast<int64_t>(share) * NC) / n_ctas);
  const int x1 = kRange && share == n_ctas ? x0 : static_cast<int>((static_cast<int64_t>(share + 1) * NC) / n_ctas);
  // With groups the grid starts beside the kernel over their prefixes, whose
  // output only the merge reads: the last CTA waits for it before it ends, and
  // with it the grid, while the others leave their SMs to the next ones.
  const bool beside = kRange && p.cu_groups != nullptr && !p.through_rep;
  if (beside && p.inline_plan && c == 0)  // the sums, for that merge
    for (int b = threadIdx.x; b <= p.B; b += blockDim.x) p.cs[b] = cs[b];
  const bool waits = beside && c == static_cast<int>(gridDim.x) - 1;
  if (x0 >= x1) {
    if (waits) pdl_wait();
    return;
  }

  uint64_t* full = reinterpret_cast<uint64_t*>(smem + p.off_bar);
  uint64_t* empty = full + kStages;
  int4* meta = reinterpret_cast<int4*>(smem + p.off_meta);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + p.off_abort);

  if (threadIdx.x == 0) {
#pragma unroll
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], NW);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  cta_sync();

  if (warp == NW) {
    // ------------------------------ producer ------------------------------
    const uint64_t pol = l2_policy_evict_first();
    const int tok = 1 << p.log2T;
    int b = kRange && p.per_request ? c : p.inline_plan ? first_request(cs, p.B, x0) : p.cta_seq[c];
    int issued = 0;
    bool aborted = false;
    for (int xg = x0; xg < x1 && !aborted; xg += 32) {
      const int nvalid = min(32, x1 - xg);
      const int x = xg + lane;
      int my_b = b, n = 0, flags = 0, new_slot = -1;
      long long off = 0;
      if (lane < nvalid) {
        while (my_b < p.B - 1 && cs[my_b - cs0 + 1] <= x) ++my_b;
        const int cb0 = cs[my_b - cs0], cb1 = cs[my_b - cs0 + 1];
        const int jc = x - cb0;
        const int L = p.ctx[my_b];
        int t0 = jc << p.log2T;
        [[maybe_unused]] Hole hole{0, 0};
        int end = L, table = my_b;
        if constexpr (kRange) {
          hole = hole_of(p, my_b, L);
          if (p.through_rep) {
            const int pre_chunks = (hole.hi + tok - 1) >> p.log2T;
            if (jc < pre_chunks) {  // of the prefix
              const int cap = static_cast<int>(min(static_cast<int64_t>(p.max_ctx), static_cast<int64_t>(p.maxp) << p.log2P));
              table = prefix_owner(p, my_b, hole.hi, cap);
              end = hole.hi;
              hole.hi = 0;
            } else {
              t0 = (jc - pre_chunks + (hole.hi >> p.log2T)) << p.log2T;
            }
          } else if (jc >= chunks_before_hole(hole, p.log2T)) {
            t0 += chunks_in_hole(hole, L, p.log2T) << p.log2T;
          }
        }
        n = min(tok, end - t0);
        const int page = p.bt[static_cast<int64_t>(table) * p.maxp + (t0 >> p.log2P)];
        if (page < 0 || page >= p.num_pages) {
          raise_flag(p.err, PA_DEVERR_BAD_PAGE);
          n = 0;
        } else {
          off = ((static_cast<long long>(page) << p.log2P) + (t0 & (p.P - 1))) * p.row_bytes;
        }
        flags = ((x == x0 || jc == 0) ? 1 : 0) | ((x == x1 - 1 || x == cb1 - 1) ? 2 : 0) |
                ((cb0 >= x0 && cb1 <= x1) ? 4 : 0) | ((x == cb1 - 1) ? 8 : 0) | ((cb1 <= x1) ? 16 : 0);
        if constexpr (kRange) {
          const int a = min(max(hole.lo - t0, 0), n), z = min(max(hole.hi - t0, 0), n);
          if (z > a) flags |= a << 8 | z << 16;
          // the keys before the range are another kernel's: this share is a part however whole it is
          if (beside && hole.hi > 0) flags &= ~4;
        }
        if (p.k_new != nullptr && (flags & 8) && n >= 1)
          new_slot = static_cast<int>(off / p.row_bytes) + n - 1;  // position context_len - 1
      }
      b = __shfl_sync(0xffffffffu, my_b, nvalid - 1);
      for (int u = 0; u < nvalid; ++u) {
        const int ub = __shfl_sync(0xffffffffu, my_b, u);
        const int un = __shfl_sync(0xffffffffu, n, u);
        const int uf = __shfl_sync(0xffffffffu, flags, u);
        const long long uoff = __shfl_sync(0xffffffffu, off, u);
        const int uslot = __shfl_sync(0xffffffffu, new_slot, u);
        int ok = 1;
        if (lane == 0) {
          const int it = xg - x0 + u;
          const int s = it % kStages;
          if (!mbar_wait_bounded(&empty[s], ((it / kStages) & 1) ^ 1, abort_flag, p.err)) {
            ok = 0;
          } else {
            meta[s] = make_int4(ub, un, uf, uslot);
            // (rows left out of a range are not copied for the tensor cores; the CUDA cores' chunk is one copy)
            const int left_out = kRange && kMma ? ((uf >> 16) & 31) - ((uf >> 8) & 31) : 0;
            const uint32_t bytes = static_cast<uint32_t>(un - left_out) * static_cast<uint32_t>(p.row_bytes);
            // tensor-core consumers read the new token's row themselves
            const uint32_t copied = kMma && uslot >= 0 ? bytes - static_cast<uint32_t>(p.row_bytes) : bytes;
            mbar_arrive_expect_tx(&full[s], 2 * copied);
            unsigned char* dst = smem + static_cast<size_t>(s) * 2 * p.chunk_bytes;
            if constexpr (kMma) {
              // the row copies are issued by the whole warp below
              if (uslot >= 0 && p.slot_out) p.slot_out[ub] = uslot;
            } else if (uslot >= 0) {
              // the cached rows of the chunk, then the new token's row from k_new / v_new
              const uint32_t cached = bytes - p.row_bytes;
              if (cached) {
                bulk_g2s_hint(dst, p.k_cache + uoff, cached, &full[s], pol);
                bulk_g2s_hint(dst + p.chunk_bytes, p.v_cache + uoff, cached, &full[s], pol);
              }
              bulk_g2s(dst + cached, p.k_new + ub * p.k_new_stride, p.row_bytes, &full[s]);
              bulk_g2s(dst + p.chunk_bytes + cached, p.v_new + ub * p.v_new_stride, p.row_bytes, &full[s]);
              if (p.slot_out) p.slot_out[ub] = uslot;
            } else if (bytes) {
              bulk_g2s_hint(dst, p.k_cache + uoff, bytes, &full[s], pol);
              bulk_g2s_hint(dst + p.chunk_bytes, p.v_cache + uoff, bytes, &full[s], pol);
            }
            if (p.k_new != nullptr && (uf & 8) && uslot < 0 && p.slot_out) p.slot_out[ub] = -1;
            ++issued;
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) {
          aborted = true;
          break;
        }
        if constexpr (kMma) {
          // one copy per token row into rows of row_pitch bytes (the pad keeps
          // the MMA consumers' fragment loads free of bank conflicts): lane r
          // copies K row r, lane 16 + r V row r; the new token's row is read
          // by the consumers from k_new / v_new
          __syncwarp();
          const int s = (xg - x0 + u) % kStages;
          unsigned char* dst = smem + static_cast<size_t>(s) * 2 * p.chunk_bytes;
          const int r = lane & 15;
          const bool isv = lane >= 16;
          const bool out = kRange && r >= ((uf >> 8) & 31) && r < ((uf >> 16) & 31);
          if (r < un && !out && !(uslot >= 0 && r == un - 1)) {
            unsigned char* d = dst + (isv ? p.chunk_bytes : 0) + r * p.row_pitch;
            const char* src = (isv ? p.v_cache : p.k_cache) + uoff + static_cast<int64_t>(r) * p.row_bytes;
            bulk_g2s_hint(d, src, p.row_bytes, &full[s], pol);
          }
        }
      }
    }
    if (aborted && lane == 0) {
      // Copies already issued may still be landing: wait for them (time only).
      for (int it = max(0, issued - kStages); it < issued; ++it)
        drain_wait(&full[it % kStages], (it / kStages) & 1);
    }
    if (waits) pdl_wait();
    return;
  }

  // ------------------------------- consumers -------------------------------
  if constexpr (kMma) {
    mma_consumer<G, kStages, kRange>(p, smem, full, empty, meta, abort_flag, x0, x1, c);
    return;
  }
  const int h = warp;
  const int rs = lane / LPR, j = lane % LPR;
  const int vbase = (j >> DUP) * VF;
  const int g_l = vbase / kTPL;          // head of the lane's kept values
  const int i_l0 = vbase % kTPL;         // token index of its first kept value
  const bool writer = (j & ((1 << DUP) - 1)) == 0;
  const bool head_leader = writer && rs == 0 && (((j >> DUP) & ((1 << IBITS) - 1)) == 0) && g_l < G;
  float* p_tile = reinterpret_cast<float*>(smem + p.off_p) + warp * Gm::TOK * PR;
  float* alpha_s = reinterpret_cast<float*>(smem + p.off_alpha) + warp * 8;
  float* ml_s = reinterpret_cast<float*>(smem + p.off_ml) + warp * 16;

  float2 qf[G][NPR];
  float2 o[G][NPR];
  float m_run = -INFINITY, l_run = 0.f;

  for (int x = x0, it = 0; x < x1; ++x, ++it) {
    const int s = it % kStages;
    if (!mbar_wait_bounded(&full[s], (it / kStages) & 1, abort_flag, p.err)) break;
    const int4 md = meta[s];
    const int b = md.x, n = md.y, flags = md.z;
    const int hole_a = kRange ? (flags >> 8) & 31 : 0, hole_z = kRange ? (flags >> 16) & 31 : 0;
    auto seen = [&](int t) { return kRange ? t < n && (t < hole_a || t >= hole_z) : t < n; };

    if (flags & 1) {  // first chunk of this CTA's share of request b
      const char* qb = p.q + (static_cast<int64_t>(b) * p.Hq + h * G) * Gm::RB + j * 16;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        float2 f[NPR];
        unpack16<T, NPR>(ldg16(qb + g * Gm::RB), f);
#pragma unroll
        for (int r = 0; r < NPR; ++r) {
          qf[g][r] = make_float2(f[r].x * p.scale_log2, f[r].y * p.scale_log2);
          o[g][r] = make_float2(0.f, 0.f);
        }
      }
      m_run = -INFINITY;
      l_run = 0.f;
    }

    const unsigned char* kbuf = smem + static_cast<size_t>(s) * 2 * p.chunk_bytes + h * Gm::RB + j * 16;
    const unsigned char* vbuf = kbuf + p.chunk_bytes;
    if (md.w >= 0) {
      // fused KV write: this head's 16-byte pieces of the new row go to its slot
      // (row slots of the warp take K and V in turn)
      const int64_t dst_off = static_cast<int64_t>(md.w) * p.row_bytes + h * Gm::RB + j * 16;
      const int src_off = (n - 1) * p.row_pitch;
      for (int part = rs; part < 2; part += RPI) {
        const unsigned char* src = (part == 0 ? kbuf : vbuf) + src_off;
        char* dst = const_cast<char*>(part == 0 ? p.k_cache : p.v_cache) + dst_off;
        stg16(dst, *reinterpret_cast<const uint4*>(src));
      }
    }

    // scores: partial dot products over this lane's 16 bytes of each row,
    // reduced over the row's lanes by a halving butterfly.  The score of
    // (head g, token i) is value g * kTPL + i, and the butterfly halves the
    // highest value bit first, so its first log2(GP) levels pair heads of one
    // token: they run per token, right after that token's products.
    float a[kTPL];
#pragma unroll
    for (int i = 0; i < kTPL; ++i) {
      const int t = i * RPI + rs;
      float2 kf[NPR];
      unpack16<T, NPR>(*reinterpret_cast<const uint4*>(kbuf + t * p.row_pitch), kf);
      float b[GP];
#pragma unroll
      for (int g = 0; g < GP; ++g) {
        if (g < G) {
          float2 acc = make_float2(0.f, 0.f);
#pragma unroll
          for (int r = 0; r < NPR; ++r) acc = ffma2(qf[g][r], kf[r], acc);
          b[g] = acc.x + acc.y;
        } else {
          b[g] = 0.f;
        }
      }
      Halve<GP, LPR / 2>::run(b, lane);
      a[i] = b[0];
    }
    if constexpr (LPR / (2 * GP) >= 1) Butterfly<kTPL, LPR / (2 * GP)>::run(a, lane);

    // online softmax (base 2) for the lane's head
    float sc[VF];
    float mc = -INFINITY;
#pragma unroll
    for (int u = 0; u < VF; ++u) {
      const int t = (i_l0 + u) * RPI + rs;
      sc[u] = seen(t) ? a[u] : -INFINITY;
      mc = fmaxf(mc, sc[u]);
    }
#pragma unroll
    for (int k = 0; k < IBITS; ++k) mc = fmaxf(mc, __shfl_xor_sync(0xffffffffu, mc, 1 << (DUP + k)));
#pragma unroll
    for (int msk = LPR; msk < 32; msk <<= 1) mc = fmaxf(mc, __shfl_xor_sync(0xffffffffu, mc, msk));
    const float m_new = fmaxf(m_run, mc);
    const float m_use = m_new == -INFINITY ? 0.f : m_new;
    const float alpha = exp2f(m_run - m_use);
    float psum = 0.f;
#pragma unroll
    for (int u = 0; u < VF; ++u) {
      const float pv = exp2f(sc[u] - m_use);
      psum += pv;
      if (writer && g_l < G)
        *reinterpret_cast<float2*>(p_tile + ((i_l0 + u) * RPI + rs) * PR + 2 * g_l) = make_float2(pv, pv);
    }
    l_run = l_run * alpha + psum;
    m_run = m_new;
    if (head_leader) alpha_s[g_l] = alpha;
    __syncwarp();

    bool rescale = false;
    float al[G];
#pragma unroll
    for (int g4 = 0; g4 < G; g4 += 4) {
      const float4 a4 = *reinterpret_cast<const float4*>(alpha_s + g4);
      const float av[4] = {a4.x, a4.y, a4.z, a4.w};
#pragma unroll
      for (int g = g4; g < G && g < g4 + 4; ++g) {
        al[g] = av[g - g4];
        rescale |= al[g] != 1.f;
      }
    }
    if (rescale) {
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int r = 0; r < NPR; ++r) o[g][r] = fmul2(o[g][r], make_float2(al[g], al[g]));
    }

    // o += p * V for this lane's 16 bytes of each row
#pragma unroll
    for (int i = 0; i < kTPL; ++i) {
      const int t = i * RPI + rs;
      if (seen(t)) {
        float2 vf[NPR];
        unpack16<T, NPR>(*reinterpret_cast<const uint4*>(vbuf + t * p.row_pitch), vf);
        const float4* prow = reinterpret_cast<const float4*>(p_tile + t * PR);
#pragma unroll
        for (int g2 = 0; g2 < G; g2 += 2) {
          const float4 pv2 = prow[g2 / 2];  // (p_g, p_g, p_g+1, p_g+1)
          const float2 pp0 = make_float2(pv2.x, pv2.y);
#pragma unroll
          for (int r = 0; r < NPR; ++r) o[g2][r] = ffma2(pp0, vf[r], o[g2][r]);
          if (g2 + 1 < G) {
            const float2 pp1 = make_float2(pv2.z, pv2.w);
#pragma unroll
            for (int r = 0; r < NPR; ++r) o[g2 + 1][r] = ffma2(pp1, vf[r], o[g2 + 1][r]);
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[s]);

    if (flags & 2) {  // last chunk of the share: write the result
#pragma unroll
      for (int msk = LPR; msk < 32; msk <<= 1)
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
          for (int r = 0; r < NPR; ++r) {
            o[g][r].x += __shfl_xor_sync(0xffffffffu, o[g][r].x, msk);
            o[g][r].y += __shfl_xor_sync(0xffffffffu, o[g][r].y, msk);
          }
      float lt = l_run;
#pragma unroll
      for (int k = 0; k < IBITS; ++k) lt += __shfl_xor_sync(0xffffffffu, lt, 1 << (DUP + k));
#pragma unroll
      for (int msk = LPR; msk < 32; msk <<= 1) lt += __shfl_xor_sync(0xffffffffu, lt, msk);
      if (head_leader) {
        ml_s[2 * g_l] = m_run;
        ml_s[2 * g_l + 1] = lt;
      }
      __syncwarp();
      if (rs == 0) {
        const bool whole = (flags & 4) != 0;
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const float mg = ml_s[2 * g], lg = ml_s[2 * g + 1];
          const float inv = lg > 0.f ? 1.f / lg : 0.f;
          const int hq = h * G + g;
          if (whole) {
            char* dst = p.out + (static_cast<int64_t>(b) * p.Hq + hq) * Gm::RB + j * 16;
            stg16(dst, pack16<T, NPR>(o[g], inv));
          } else {
            const int64_t slot = static_cast<int64_t>(c) + b;
            float* dst = p.o_part + (slot * p.Hq + hq) * HD + j * Gm::DPL;
#pragma unroll
            for (int r = 0; r < NPR; r += 2)
              *reinterpret_cast<float4*>(dst + 2 * r) =
                  make_float4(o[g][r].x * inv, o[g][r].y * inv, o[g][r + 1].x * inv, o[g][r + 1].y * inv);
            if (j == 0) p.lse_part[slot * p.Hq + hq] = (kRange ? lg != 0.f : lg > 0.f) ? mg + log2f(lg) : -INFINITY;
          }
        }
      }
      __syncwarp();
    }
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
struct Fns {
  const void* main = nullptr;
  const void* merge = nullptr;
};

template <bool kRange, typename T, int HD>
Fns fns_for_g(int G) {
  const void* merge = reinterpret_cast<const void*>(decode_merge_kernel<T, HD, kRange>);
  switch (G) {
    case 1: return {reinterpret_cast<const void*>(decode_kernel<T, HD, 1, kRange>), merge};
    case 2: return {reinterpret_cast<const void*>(decode_kernel<T, HD, 2, kRange>), merge};
    case 3: return {reinterpret_cast<const void*>(decode_kernel<T, HD, 3, kRange>), merge};
    case 4: return {reinterpret_cast<const void*>(decode_kernel<T, HD, 4, kRange>), merge};
    case 5: return {reinterpret_cast<const void*>(decode_kernel<T, HD, 5, kRange>), merge};
    case 6: return {reinterpret_cast<const void*>(decode_kernel<T, HD, 6, kRange>), merge};
    case 7: return {reinterpret_cast<const void*>(decode_kernel<T, HD, 7, kRange>), merge};
    case 8: return {reinterpret_cast<const void*>(decode_kernel<T, HD, 8, kRange>), merge};
    default: return {};
  }
}

template <bool kRange>
Fns get_fns(int dtype, int hd, int G) {
  if (dtype == PA_BF16)
    return hd == 128 ? fns_for_g<kRange, __nv_bfloat16, 128>(G) : fns_for_g<kRange, __nv_bfloat16, 64>(G);
  return hd == 128 ? fns_for_g<kRange, float, 128>(G) : fns_for_g<kRange, float, 64>(G);
}

bool uses_mma(int dtype, int hd, int /*G*/) { return dtype == PA_BF16 && hd == 128; }

// The plan of a batch whose requests have up to max_ctx keys, of which up to
// max_keys, in up to `extra` chunks more than those would fill, are attended to.
template <bool kRange>
cudaError_t plan_decode_keys(const pa_cache_desc& d, int batch, int max_ctx, int max_keys, int extra, int max_ctas,
                             DecodePlan* out) {
  DeviceInfo di;
  cudaError_t e = current_device_info(&di);
  if (e != cudaSuccess) return e;
  const int E = elem_bytes(d.dtype);
  const int G = d.num_q_heads / d.num_kv_heads;
  const Fns f = get_fns<kRange>(d.dtype, d.head_dim, G);
  if (!f.main) return cudaErrorInvalidValue;
  const int dpl = 16 / E, lpr = d.head_dim / dpl, rpi = 32 / lpr;
  DecodePlan pl;
  pl.nw = d.num_kv_heads;
  pl.tokens_per_chunk = uses_mma(d.dtype, d.head_dim, G) ? kMmaTok : kTPL * rpi;
  const int row_bytes = d.num_kv_heads * d.head_dim * E;
  pl.row_pitch = uses_mma(d.dtype, d.head_dim, G) ? row_bytes + 16 : row_bytes;
  pl.chunk_bytes = pl.tokens_per_chunk * pl.row_pitch;
  const int stages = uses_mma(d.dtype, d.head_dim, G) ? kStagesMma : kStages;
  pl.stages = stages;
  size_t off = static_cast<size_t>(stages) * 2 * pl.chunk_bytes;
  pl.off_bar = static_cast<uint32_t>(off);
  off += 2 * stages * sizeof(uint64_t);
  pl.off_meta = static_cast<uint32_t>(align_up(off, 16));
  off = pl.off_meta + stages * 16;
  pl.off_abort = static_cast<uint32_t>(off);
  off += 16;
  pl.p_row = p_row_floats(G);
  pl.off_p = static_cast<uint32_t>(align_up(off, 16));
  off = pl.off_p + static_cast<size_t>(pl.nw) * pl.tokens_per_chunk * pl.p_row * 4;
  pl.off_alpha = static_cast<uint32_t>(align_up(off, 16));
  off = pl.off_alpha;
  off += static_cast<size_t>(pl.nw) * 8 * 4;
  pl.off_ml = static_cast<uint32_t>(off);
  off += static_cast<size_t>(pl.nw) * 16 * 4;
  // room for the batch's prefix sums (whatever the batch, so that the CTAs
  // per SM, and with them the plan, do not depend on it)
  pl.off_cs = static_cast<uint32_t>(align_up(off, 16));
  off = pl.off_cs + static_cast<size_t>(kInlinePlanMax + 1 + 32) * 4;
  pl.smem_bytes = align_up(off, 128);
  if (pl.smem_bytes > static_cast<size_t>(di.max_smem_optin)) return cudaErrorInvalidValue;
  int occ = 0;
  e = ctas_per_sm(di, f.main, (pl.nw + 1) * 32, pl.smem_bytes, &occ);
  if (e != cudaSuccess) return e;
  const int64_t T = pl.tokens_per_chunk;
  const int64_t chunks_upper = batch * std::min((max_ctx + T - 1) / T, (max_keys + T - 1) / T + extra);
  pl.slots = occ * di.sm_count;
  int64_t n = pl.slots;
  if (max_ctas > 0) n = std::min<int64_t>(n, max_ctas);
  n = std::min<int64_t>(n, std::max<int64_t>(1, chunks_upper));
  pl.n_ctas = static_cast<int>(std::max<int64_t>(1, n));
  decode_workspace_layout(d, batch, &pl);
  *out = pl;
  return cudaSuccess;
}

}  // namespace
}  // namespace pa
