// Batched GQA decode attention over a 4-bit paged cache (sm_103a).
//
// The mathematics is decode.cu's over the values that K and V rows of 4-bit codes
// stand for (q4_common.cuh): the even split of the keys over the CTAs, the partial
// results and their merge are the same code (decode_shared.cuh).  A chunk is
// 32 tokens, two halves of 16 tokens of one page each; a producer warp copies
// their rows of K and V as they are into a ring in shared memory (one run of
// rows where the halves follow each other in a page), and one consumer warp
// per kv-head takes its head's part.
//
// The floor is HBM's; over a call's life the kernel does not reach it.  Measured
// (16-bit queries, 8 kv-heads of 128 dims; the call with its merge, replayed from a
// graph): 256 requests of 128-2048 tokens, groups of 32, 72.3 us for 347 MB; 64 of
// 1024-8192, groups of 64, 67.1 us for 355 MB; 8 of 32768, groups of 128, 56.2 us for
// 285 MB: 4.8 to 5.3 TB/s of a copy's 6.7.  Of these the start (plan, page look-up,
// first chunk) takes 6 to 7 and the merge 2 to 4 us.
#include "decode_shared.cuh"
#include "q4_common.cuh"

namespace pa {
namespace {

constexpr int kTok = 32;        // tokens per chunk
constexpr int kHalf = 16;       // tokens of a half chunk (a page holds whole halves)
constexpr int kMaxStages = 8;   // ring depth, at most
constexpr int kMaxCluster = 8;  // CTAs of a cluster that shares a request, at most
// Tokens of 128 dims (of 64 twice as many; fp32, which takes a token about half as
// fast, half as many) of a request that a CTA takes, alone or with its cluster, where
// a CTA or a cluster per request comes to at least 2/5 of the SMs; and that a CTA
// alone takes in any batch.
constexpr int kPartTokens = 256, kAloneTokens = 64;

// A chunk in the ring, as the producer describes it to the consumers: its
// request; the tokens of its halves (n0 | n1 << 8, 0 for a half whose page is
// out of range) and flags; the share it belongs to; and the slot of the
// request's new token when it is the last of these tokens (else -1).
constexpr uint32_t kFirst = 1u << 16;  // the consumer group's first chunk of the request: the queries come with it
constexpr uint32_t kLast = 1u << 17;   // the share's last chunk of the request: its group writes the result
constexpr uint32_t kYield = 1u << 18;  // the other group's last chunk of the request: it hands its part over
constexpr uint32_t kSolo = 1u << 19;   // with kLast: the other group has no part
constexpr uint32_t kWhole = 1u << 20;  // the share holds the whole request
constexpr uint32_t kRagged = 1u << 21; // a half has fewer than 16 tokens
constexpr uint32_t kNew = 1u << 22;    // the request's new token is the last one
constexpr uint32_t kEnd = 1u << 23;    // no chunk: the CTA's work is done
constexpr uint32_t kSettle = 1u << 24; // every kSettleChunks-th of a consumer group's chunks of the request

constexpr int kSettleChunks = 8;  // bf16: chunks whose second term is summed apart

struct Q4Params {
  KParams k;
  int32_t stages;       // ring depth
  int32_t stage_bytes;  // K rows, V rows, queries
  int32_t groups;       // consumer groups: 2 (bf16) or 1 (fp32)
  int32_t cluster;      // CTAs of each request; 0: the CTAs share the batch's chunks evenly
  uint32_t off_hand;    // [Hq][HD + 4] fp32: the part that one group hands to the other, or a CTA to its cluster
  int32_t codes, pars;  // bytes of the two parts of a row
  int32_t log2gs;
};

// The row of a 4-bit cache.
template <int HD, int NG, int HKV>
struct Q4Row {
  static constexpr uint32_t kCodes = HKV * HD / 2;
  static constexpr uint32_t kPars = (HKV * NG * 4 + 15) / 16 * 16;
  static constexpr uint32_t kBytes = kCodes + kPars;
};

// Position in the ring: stage and phase bit of the running chunk.
struct Ring {
  int s = 0;
  uint32_t phase = 0;
  PA_DEVINL void next(int stages) {
    if (++s == stages) {
      s = 0;
      phase ^= 1;
    }
  }
  PA_DEVINL void next2(int stages) {
    s += 2;
    if (s >= stages) {
      s -= stages;
      phase ^= 1;
    }
  }
};

// The new token's K and V of kv-head h, quantised by the warp: into row t of the
// chunk's stage and into the cache.  Every lane takes eight dims: K in the
// lower lanes, V behind it.
template <typename T, int HD>
PA_DEVINL void write_new_row(const Q4Params& p, unsigned char* kst, unsigned char* vst, int b, uint32_t t, int slot,
                             int h, int lane) {
  constexpr int LPR = HD / 8;
  const bool isv = (lane / LPR) & 1;
  const int l = lane % LPR;
  const char* src = (isv ? p.k.v_new + static_cast<int64_t>(b) * p.k.v_new_stride
                         : p.k.k_new + static_cast<int64_t>(b) * p.k.k_new_stride) +
                    (h * HD + l * 8) * sizeof(T);
  uint32_t words[kQ4Words<T>];
  q4_load8<T>(src, words);
  const int gl = 1 << (p.log2gs - 3);
  uint32_t par;
  const uint32_t w = q4_quantise8<T>(words, gl, par);
  if (lane < 2 * LPR) {
    unsigned char* row = (isv ? vst : kst) + t * p.k.row_bytes;
    char* dst = const_cast<char*>(isv ? p.k.v_cache : p.k.k_cache) + static_cast<int64_t>(slot) * p.k.row_bytes;
    const uint32_t co = q4_swz(h * (HD / 2) + l * 4, p.codes, t);
    *reinterpret_cast<uint32_t*>(row + co) = w;
    *reinterpret_cast<uint32_t*>(dst + co) = w;
    if ((l & (gl - 1)) == 0) {
      const uint32_t po = p.codes + q4_swz((h * (HD >> p.log2gs) + ((l * 8) >> p.log2gs)) * 4, p.pars, t);
      *reinterpret_cast<uint32_t*>(row + po) = par;
      *reinterpret_cast<uint32_t*>(dst + po) = par;
    }
  }
  // the fence orders these stores before the copies that refill the stage later
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
}

// log2-sum-exp of a partial result.  One without tokens (all on bad pages) has no
// weight in a merge; one that is not a number has all of it.
PA_DEVINL float partial_lse(float m, float l) { return l > 0.f ? m + log2f(l) : l == 0.f ? -INFINITY : INFINITY; }

// ---------------------------------------------------------------------------
// Consumer (groups of up to 8 q-heads).
//
// Per chunk, S^T = K Q^T and O^T += V^T P^T as mma.sync m16n8k16 (float16 in,
// fp32 out): 16 tokens, then 16 of the head's dims, are the rows, and the
// group's q-heads the 8 columns (heads past G are zero queries), so no row of a
// product is padding.  With l = 4 gq + tq, a lane holds of A rows gq and gq + 8
// at columns 2 tq, 2 tq + 1 (+ 8), of B column gq at rows 2 tq, 2 tq + 1 (+ 8),
// of C rows gq and gq + 8 at columns 2 tq, 2 tq + 1 (PTX ISA).
//
// Neither the order of the dims inside a sum nor that of O's rows matters to the
// result, so a lane's share is what ldmatrix hands it of 16-byte pieces, 32 dims
// of a token each (the pieces of eight consecutive tokens lie in different banks,
// whatever the row's size): of K, word tq of tokens gq and gq + 8, eight dims of
// which a register pairs d and d + 4; of V, transposed, half word gq of tokens
// 2 tq, 2 tq + 1 (+ 8), four dims that each pair two tokens in a register.
//
// The kernel is bound by instructions, not bytes, until decoding is cheap, so
// codes enter the products undecoded: u in bits 6-9 (2-5) of a half word is the
// subnormal float16 u * 2^-18 (2^-22), exact, one mask.  With m = 16 s + c the
// value is s u + m, so
//   S = sum over groups of s (sum q u) + m (sum q):  the sums of q u are scaled
//       by s as they leave the tensor cores, the second term is one product of the
//       parameter words (s, c) with (16 sum q, sum q), each sum as two float16
//       numbers;
//   O = sum over tokens of (p s) u + p m:  p s replaces p as the B operand, and
//       the second term is one product of the transposed parameter piece, whose
//       rows are its groups' s and c, with p.  The product's other eight rows
//       are ones: the softmax sum.  Every 256 tokens of a group of consumers
//       (kSettle) the second term joins O: apart, the two sums grow with the tokens,
//       what the tensor cores cut off of them with the square, and it stays when the
//       two all but cancel (4% of outputs whose values have no mean at 100000
//       tokens; together 0.2%, the output's rounding; at 2048 and below no change).
// 16 tokens of a head take 212 instructions with groups of 128, 113 of them on
// the integer pipe (two cycles each), 256 with groups of 32 (fp32: 383 and 709);
// 309 with K and V decoded to float16 in registers, 228 with raw codes loaded as
// words and paired by byte permutes.
//
// fp32 queries and outputs.  Queries and p s are two float16 numbers each, multiples
// of 2^-11 and 2^-23 of their bounds, so that every sum of products with codes is
// exact; the two sums and those of 16 tokens are added in fp32.  The bounds are those
// of a head's group of dims (p s: among 16 tokens): keys of one group may be far
// smaller than another's, and a query that is large there must not coarsen the rest
// (with one bound for a head, outputs were off by 1e-4 where queries of one group were
// 2^10 times the others' and its keys as much smaller).  The second terms and the
// softmax sum are fp32 multiply-adds of the lanes: the terms cancel to a fifth or less,
// and what a tensor core's additions cut off (1e-7 of the largest) would show.  For the
// same reason the 16 tokens' p m join their p s u before either enters O: summed apart
// over a share the two grow with its tokens, their difference with the root of these,
// and it kept their rounding (2.9e-4 of the outputs at 20000 tokens; now 3e-6).  One
// consumer group, whose warps may have 168 registers.
//
// Ranges.  Queries are scaled by a power of two to a largest magnitude in [2^8, 2^9)
// (of the head; fp32: of each group).  A head's largest probability lies between 2^7 and
// 2^11 (their reference follows the maximum when a score passes it by more).  p s is kept
// in float16's range by a power of two 2^-E that follows the largest s seen in the share:
// s has all its bits down to 2^-18 of that, p s while weight times s is at least 2^-25 of
// the largest weight times the largest s.  Each rounding to float16 is 2^-11 relative,
// finer than the bf16 of queries and outputs; sums and statistics are fp32.
// ---------------------------------------------------------------------------
PA_DEVINL void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// d = A (B0 + B1) with 8 columns of A.
PA_DEVINL void mma_f16_twice(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %4, %5}, {%6, %7}, "
      "{%8, %8, %8, %8};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(b0), "r"(b1), "f"(0.f));
}

// Transpose of an 8x8 matrix of 16-bit elements held two to a lane.
PA_DEVINL uint32_t movm_trans(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

PA_DEVINL uint32_t pack_f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

PA_DEVINL uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

PA_DEVINL float f16_lo(uint32_t w) { return __half2float(__ushort_as_half(static_cast<uint16_t>(w & 0xFFFFu))); }

// A head's largest probability is 2^7 at first and at most 2^11, and s at most 2^5, so
// that p s is a float16.  Probabilities down to 2^-21 of the largest have all of its
// bits, and 2^20 tokens lose no more than 2^-12 of their weight to those below 2^-32.
constexpr float kFirstMost = 7.f, kMost = 11.f;
constexpr uint32_t kOnes = 0x3C003C00u;      // 1 twice
constexpr uint32_t kExponent = 0x04000400u;  // the lowest exponent bit of a float16, twice

// u * 2^-18 of the codes in bits 6-9, u * 2^-22 of those in bits 2-5.
PA_DEVINL uint32_t raw_hi(uint32_t w) { return w & 0x03C003C0u; }
PA_DEVINL uint32_t raw_lo(uint32_t w) { return w & 0x003C003Cu; }

// mbarriers by their shared-memory address: the consumers' registers are scarce,
// and 64-bit pointers to them would take a dozen.
PA_DEVINL bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// As mbar_wait_bounded, with the abort flag at a shared-memory address.
PA_DEVINL bool bar_wait_slow(uint32_t bar, uint32_t parity, uint32_t abort, unsigned int* err) {
  const uint64_t t0 = global_timer_ns();
  for (uint32_t it = 1;; ++it) {
    if (bar_try(bar, parity)) return true;
    if ((it & 63u) == 0) {
      uint32_t gone;
      asm volatile("ld.volatile.shared.b32 %0, [%1];" : "=r"(gone) : "r"(abort) : "memory");
      if (gone) return false;
      if (global_timer_ns() - t0 > kWaitLimitNs) {
        asm volatile("st.volatile.shared.b32 [%0], %1;" ::"r"(abort), "r"(1u) : "memory");
        raise_flag(err, PA_DEVERR_TIMEOUT);
        return false;
      }
    }
  }
}

PA_DEVINL bool bar_wait(uint32_t bar, uint32_t parity, uint32_t abort, unsigned int* err) {
  return bar_try(bar, parity) || bar_wait_slow(bar, parity, abort, err);
}

PA_DEVINL void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Loads from a shared-memory address.  Volatile: they stay between the wait for
// a stage and its release.
PA_DEVINL uint32_t lds32(uint32_t a) {
  uint32_t r;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r) : "r"(a));
  return r;
}
// N consecutive words.
template <int N>
PA_DEVINL void lds_words(uint32_t* r, uint32_t a) {
  static_assert(N == 1 || N == 2 || N == 4, "");
  if constexpr (N == 1) {
    r[0] = lds32(a);
  } else if constexpr (N == 2) {
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(a));
  } else {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
  }
}

// Four 8x8 matrices of 16-bit elements, lane i's address that of row i % 8 of
// matrix i / 8: two elements of row lane / 4 each, or (trans) of column lane / 4.
PA_DEVINL void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
PA_DEVINL void ldsm4_trans(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}

// x = hi + lo + less than 2^-12 of kGrid: hi a multiple of kGrid, lo of 2^-12
// kGrid, both float16 numbers where |x| <= 2^11 kGrid.
template <int kLog2Grid>
PA_DEVINL void split(float x, float& hi, float& lo) {
  constexpr float m = 1.5f * (1 << 23), g = kLog2Grid < 0 ? 1.f / (1 << -kLog2Grid) : 1.f * (1 << kLog2Grid);
  hi = __fsub_rn(__fadd_rn(x, m * g), m * g);
  const float rest = x - hi;
  lo = __fsub_rn(__fadd_rn(rest, m * g * 0x1p-12f), m * g * 0x1p-12f);
}

template <typename T, int HD, int NG, int HKV>
PA_DEVINL void consume(const Q4Params& p, unsigned char* smem, int h, int group) {
  constexpr int NP = HD / 32;          // pieces of a head's codes in a row: 32 dims each
  constexpr int PG = NP / NG;          // of them, a group's
  constexpr int MB = HD / 16;          // 16-dim blocks of O: two to a piece
  constexpr bool kF32 = sizeof(T) == 4;
  using Row = Q4Row<HD, NG, HKV>;
  constexpr uint32_t R = Row::kBytes, kChunk = kTok * R;
  const int lane = threadIdx.x & 31;
  const int G = p.k.Hq / HKV;
  const int gq = lane >> 2, tq = lane & 3;
  // Places in a stage.  Codes: this lane's row of the matrices that one load
  // takes, tokens 0-7 and 8-15 of pieces i, i + 1 (K's; V's are kChunk on).
  uint32_t c_at[NP / 2];
#pragma unroll
  for (int i = 0; i < NP / 2; ++i)
    c_at[i] = (lane & 15) * R + q4_swz(h * (HD / 2) + (2 * i + (lane >> 4)) * 16, Row::kCodes, lane);
  // K's parameters of token gq, and the piece with the head's V parameters of token `lane`
  const uint32_t kp_at = gq * R + Row::kCodes + q4_swz(h * NG * 4, Row::kPars, gq);
  const uint32_t vp_at = kChunk + lane * R + Row::kCodes + q4_swz(h * NG * 4 & ~15, Row::kPars, lane);
  // The piece's half words, rows of the transposed matrix: those of this head from
  // 2 (h NG mod 4) on, s and c of each group.  s of group g is with lanes s_lane + 8 g.
  const int s_row = h * NG % 4 * 2, s_lane = s_row * 4 + tq;
  const uint32_t s_mask = gq >= s_row && gq < s_row + 2 * NG && gq % 2 == 0 ? 0xFFFFFFFFu : 0u;
  const uint32_t smem0 = smem_u32(smem);
  // the barriers of the table in the kernel below
  auto full = [&](int s) { return smem0 + p.k.off_bar + 8 * s; };
  auto empty = [&](int s) { return smem0 + p.k.off_bar + 8 * (kMaxStages + s); };
  auto handed = [&] { return smem0 + p.k.off_bar + 8 * (2 * kMaxStages + h); };
  auto taken = [&] { return smem0 + p.k.off_bar + 8 * (2 * kMaxStages + 8 + h); };
  auto wait = [&](uint32_t bar, uint32_t parity) { return bar_wait(bar, parity, smem0 + p.k.off_abort, p.k.err); };

  uint32_t qf[MB][2];  // B fragments of the queries: 2^8 q where codes are at bits 6-9, 2^12 q where at 2-5
  [[maybe_unused]] uint32_t qm[2] = {};            // 2^2 (16 sum q, sum q) over the dims of group tq, and what it lacks
  [[maybe_unused]] uint32_t ql[kF32 ? MB : 1][2];  // fp32: what qf lacks,
  [[maybe_unused]] float q_sum[NG][2];             // and the sums, times mult, for heads 2 tq and 2 tq + 1
  [[maybe_unused]] float l_sum[2] = {0.f, 0.f};  // fp32: this lane's share of the sum over the tokens of p
  float o[MB][4];
  // Sums over the tokens: [0..1] of p s or p c (row gq of the parameter piece),
  // [2..3] of p (the softmax sums of heads 2 tq, 2 tq + 1).
  float om[4] = {0.f, 0.f, 0.f, 0.f};
  // The largest s with the exponent of the largest seen, twice (0: none above 0
  // yet).  With that exponent's bits x, E = max(x - 19, -15).  (Not for fp32.)
  uint32_t s_most = 0u;
  // score scale of heads 2 tq, 2 tq + 1 (base 2, the powers of two undone); fp32: of each group
  float mult[kF32 ? NG : 1][2];
  float m[2] = {0.f, 0.f};     // the exponents' reference of the two heads
  float limit = -INFINITY;     // scores above the reference by more than this move it: any at first, then kMost
  uint32_t hand_phase = 0;     // parity of the handovers so far
  Ring ring;
  if (group) ring.next(p.stages);  // group g takes stages g, g + 2, ... of the ring
  for (;; kF32 ? ring.next(p.stages) : ring.next2(p.stages)) {
    const int s = ring.s;
    if (!wait(full(s), ring.phase)) break;
    const uint32_t md = smem0 + p.k.off_meta + s * 16;  // {request, tokens and flags, share, slot}
    const uint32_t flags = lds32(md + 4);
    const uint32_t st = smem0 + s * p.stage_bytes;

    if (flags & (kFirst | kNew | kEnd)) {
      if (flags & kEnd) break;
      if (flags & kFirst) {
        const uint32_t qrow = st + 2 * kChunk + (h * G + gq) * HD * sizeof(T);
        float qv[NP][8];  // eight dims of each piece
        float mx[kF32 ? NG : 1] = {};
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          uint32_t w[8] = {};
          const uint32_t at = qrow + (i * 32 + tq * 8) * sizeof(T);
          if (gq < G) {
            lds_words<4>(w, at);
            if constexpr (kF32) lds_words<4>(w + 4, at + 16);
          }
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            if constexpr (kF32) {
              qv[i][e] = __uint_as_float(w[e]);
              qv[i][e + 1] = __uint_as_float(w[e + 1]);
            } else {
              const float2 v = bf16x2_to_float2(w[e / 2]);
              qv[i][e] = v.x;
              qv[i][e + 1] = v.y;
            }
            float& most = mx[kF32 ? i / PG : 0];
            most = fmaxf(most, fmaxf(fabsf(qv[i][e]), fabsf(qv[i][e + 1])));
          }
        }
        // 2^-E of the largest magnitude's exponent E (fp32: of each group's), and 2^E
        float down[kF32 ? NG : 1];
#pragma unroll
        for (int g = 0; g < (kF32 ? NG : 1); ++g) {
          mx[g] = fmaxf(mx[g], __shfl_xor_sync(0xffffffffu, mx[g], 1));
          mx[g] = fmaxf(mx[g], __shfl_xor_sync(0xffffffffu, mx[g], 2));
          const uint32_t eb = min(max(__float_as_uint(mx[g]) >> 23, 1u), 253u);
          down[g] = __uint_as_float((254u - eb) << 23);
          const float up = __uint_as_float(eb << 23) * p.k.scale_log2;
          mult[g][0] = __shfl_sync(0xffffffffu, up, 8 * tq) * 1024.f;
          mult[g][1] = __shfl_sync(0xffffffffu, up, 8 * tq + 4) * 1024.f;
        }
        qm[0] = qm[1] = 0u;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          float sum = 0.f;
          [[maybe_unused]] float sum_l = 0.f;  // (apart: the sum of the first parts is all but exact)
#pragma unroll
          for (int i = g * PG; i < (g + 1) * PG; ++i) {
            float (&q)[8] = qv[i];
            [[maybe_unused]] float l[8];
            // as they are rounded: the second term's sum has to be that of the first's queries
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float x = q[e] * down[kF32 ? g : 0] * 256.f;  // below 2^9
              if constexpr (kF32) {
                split<-2>(x, q[e], l[e]);
                sum_l += l[e];
              } else {
                q[e] = __half2float(__float2half_rn(x));
              }
              sum += q[e];
            }
            qf[2 * i][0] = pack_f16x2(q[0], q[4]);
            qf[2 * i][1] = pack_f16x2(q[1], q[5]);
            qf[2 * i + 1][0] = pack_f16x2(q[2] * 16.f, q[6] * 16.f);
            qf[2 * i + 1][1] = pack_f16x2(q[3] * 16.f, q[7] * 16.f);
            if constexpr (kF32) {
              ql[2 * i][0] = pack_f16x2(l[0], l[4]);
              ql[2 * i][1] = pack_f16x2(l[1], l[5]);
              ql[2 * i + 1][0] = pack_f16x2(l[2] * 16.f, l[6] * 16.f);
              ql[2 * i + 1][1] = pack_f16x2(l[3] * 16.f, l[7] * 16.f);
            }
          }
          sum += __shfl_xor_sync(0xffffffffu, sum, 1);
          sum += __shfl_xor_sync(0xffffffffu, sum, 2);
          if constexpr (kF32) {
            sum_l += __shfl_xor_sync(0xffffffffu, sum_l, 1);
            sum_l += __shfl_xor_sync(0xffffffffu, sum_l, 2);
            sum += sum_l;
            q_sum[g][0] = __shfl_sync(0xffffffffu, sum, 8 * tq) * 0x1p-18f * mult[g][0];
            q_sum[g][1] = __shfl_sync(0xffffffffu, sum, 8 * tq + 4) * 0x1p-18f * mult[g][1];
          } else {
            // (at most 2^10; the second term is as large as the first for keys with a mean)
            const float r = __half2float(__float2half_rn(sum * 0x1p-6f)), rest = sum * 0x1p-6f - r;
            if (tq == g) {
              qm[0] = pack_f16x2(r * 16.f, r);
              qm[1] = pack_f16x2(rest * 16.f, rest);
            }
          }
        }
#pragma unroll
        for (int j = 0; j < MB; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
        m[0] = m[1] = 0.f;
        limit = -INFINITY;
        om[0] = om[1] = om[2] = om[3] = 0.f;
        l_sum[0] = l_sum[1] = 0.f;
        s_most = 0u;
      }
      if (flags & kNew) {
        unsigned char* kst = smem + static_cast<size_t>(s) * p.stage_bytes;
        const uint32_t n0 = flags & 255, n1 = (flags >> 8) & 255;
        write_new_row<T, HD>(p, kst, kst + kChunk, lds32(md), n1 ? kHalf + n1 - 1 : n0 - 1,
                                         lds32(md + 12), h, lane);
      }
    }

    // S^T = K Q^T of both halves
    float t[2][4];
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const uint32_t half = st + hf * kHalf * R;
      uint32_t par[2][NG];  // parameters of tokens gq, gq + 8
#pragma unroll
      for (int u = 0; u < 2; ++u) lds_words<NG>(par[u], half + u * 8 * R + kp_at);
      float sc[4] = {0.f, 0.f, 0.f, 0.f}, d[4];
      [[maybe_unused]] float dl[4];  // fp32: of the lower parts of the queries
      if constexpr (!kF32) {
        uint32_t pm[2];  // of their group tq (any where there is none: its queries' sum is 0)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          pm[u] = par[u][0];
          if constexpr (NG == 2) pm[u] = (tq & 1) ? par[u][1] : par[u][0];
          if constexpr (NG == 4)
            pm[u] = (tq & 2) ? ((tq & 1) ? par[u][3] : par[u][2]) : ((tq & 1) ? par[u][1] : par[u][0]);
        }
        mma_f16_twice(sc, pm[0], pm[1], qm[0], qm[1]);
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[e] *= 0x1p-12f;
      }
      uint32_t w[4];  // of two pieces: the words of tokens gq and gq + 8
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        if (i % 2 == 0) ldsm4(w, half + c_at[i / 2]);
        const uint32_t w0 = i % 2 == 0 ? w[0] : w[2], w1 = i % 2 == 0 ? w[1] : w[3];
        const uint32_t y0 = __byte_perm(w0, 0, 0x2301), y1 = __byte_perm(w1, 0, 0x2301);
        if (i % PG == 0) d[0] = d[1] = d[2] = d[3] = 0.f;
        if constexpr (kF32) {
          if (i % PG == 0) dl[0] = dl[1] = dl[2] = dl[3] = 0.f;
          mma_f16(dl, raw_hi(w0), raw_hi(w1), raw_hi(y0), raw_hi(y1), ql[2 * i][0], ql[2 * i][1]);
          mma_f16(dl, raw_lo(w0), raw_lo(w1), raw_lo(y0), raw_lo(y1), ql[2 * i + 1][0], ql[2 * i + 1][1]);
        }
        mma_f16(d, raw_hi(w0), raw_hi(w1), raw_hi(y0), raw_hi(y1), qf[2 * i][0], qf[2 * i][1]);
        mma_f16(d, raw_lo(w0), raw_lo(w1), raw_lo(y0), raw_lo(y1), qf[2 * i + 1][0], qf[2 * i + 1][1]);
        if (i % PG == PG - 1) {
          const float s0 = f16_lo(par[0][i / PG]), s1 = f16_lo(par[1][i / PG]);
          if constexpr (kF32) {
            const float m0 = fmaf(16.f, s0, f16_lo(par[0][i / PG] >> 16));
            const float m1 = fmaf(16.f, s1, f16_lo(par[1][i / PG] >> 16));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              d[e] += dl[e];
              sc[e] = fmaf(e < 2 ? m0 : m1, q_sum[i / PG][e & 1], sc[e]);
              sc[e] = fmaf(d[e], (e < 2 ? s0 : s1) * mult[i / PG][e & 1], sc[e]);
            }
          } else {
            sc[0] = fmaf(d[0], s0, sc[0]);
            sc[1] = fmaf(d[1], s0, sc[1]);
            sc[2] = fmaf(d[2], s1, sc[2]);
            sc[3] = fmaf(d[3], s1, sc[3]);
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) t[hf][e] = kF32 ? sc[e] - m[e & 1] : fmaf(sc[e], mult[0][e & 1], -m[e & 1]);
    }

    // softmax: exponents relative to a reference that lies kFirstMost below the first
    // maximum and moves up to kFirstMost below a score that passes it by more than kMost
    if (flags & kRagged) {
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int n = (flags >> (8 * hf)) & 255;
        if (gq >= n) t[hf][0] = t[hf][1] = -INFINITY;
        if (gq + 8 >= n) t[hf][2] = t[hf][3] = -INFINITY;
      }
    }
    float d0 = fmaxf(fmaxf(t[0][0], t[0][2]), fmaxf(t[1][0], t[1][2]));
    float d1 = fmaxf(fmaxf(t[0][1], t[0][3]), fmaxf(t[1][1], t[1][3]));
    if (__any_sync(0xffffffffu, fmaxf(d0, d1) > limit)) {
#pragma unroll
      for (int k = 4; k < 32; k <<= 1) {
        d0 = fmaxf(d0, __shfl_xor_sync(0xffffffffu, d0, k));
        d1 = fmaxf(d1, __shfl_xor_sync(0xffffffffu, d1, k));
      }
      if (limit == -INFINITY) {  // the first scores: O and l are zero
        d0 = d0 == -INFINITY ? 0.f : d0 - kFirstMost;
        d1 = d1 == -INFINITY ? 0.f : d1 - kFirstMost;
      } else {
        d0 = fmaxf(d0 - kFirstMost, 0.f);
        d1 = fmaxf(d1 - kFirstMost, 0.f);
        const float a0 = ex2_approx(-d0), a1 = ex2_approx(-d1);
        om[0] *= a0;
        om[1] *= a1;
        om[2] *= a0;
        om[3] *= a1;
        if constexpr (kF32) {
          l_sum[0] *= a0;
          l_sum[1] *= a1;
        }
#pragma unroll
        for (int j = 0; j < MB; ++j) {
          o[j][0] *= a0;
          o[j][1] *= a1;
          o[j][2] *= a0;
          o[j][3] *= a1;
        }
      }
      m[0] += d0;
      m[1] += d1;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        t[hf][0] -= d0;
        t[hf][1] -= d1;
        t[hf][2] -= d0;
        t[hf][3] -= d1;
      }
      limit = kMost;
    }
    uint32_t pb[2][2];  // B fragments of the probabilities
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const float p0 = ex2_approx(t[hf][0]), p1 = ex2_approx(t[hf][1]);
      const float p2 = ex2_approx(t[hf][2]), p3 = ex2_approx(t[hf][3]);
      if constexpr (kF32) {
        t[hf][0] = p0, t[hf][1] = p1, t[hf][2] = p2, t[hf][3] = p3;
      } else {
        pb[hf][0] = movm_trans(pack_f16x2(p0, p1));
        pb[hf][1] = movm_trans(pack_f16x2(p2, p3));
      }
    }

    // O^T += V^T P^T
    [[maybe_unused]] uint32_t vm[4];  // row gq of the parameter piece: tokens 2 tq, 2 tq + 1 (+ 8, + 16, + 24)
    [[maybe_unused]] uint32_t vpar[2][2][NG];  // fp32: the parameters of tokens gq, gq + 8 (+ 16)
    if constexpr (kF32) {
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          lds_words<NG>(vpar[hf][u], st + kChunk + (hf * kHalf + u * 8) * R + kp_at);
          // rows past the context meet probability 0 and must be finite
          const bool live = gq + u * 8 < static_cast<int>((flags >> (8 * hf)) & 255);
#pragma unroll
          for (int g = 0; g < NG; ++g)
            if (!live) vpar[hf][u][g] = 0u;
        }
    } else {
      ldsm4_trans(vm, st + vp_at);
      if (flags & kRagged) {
        // rows past the context meet probability 0 and must be finite
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int n = static_cast<int>((flags >> (u / 2 * 8)) & 255) - (u & 1) * 8;
          vm[u] &= (2 * tq < n ? 0xFFFFu : 0u) | (2 * tq + 1 < n ? 0xFFFF0000u : 0u);
        }
      }
      // A larger s than the scale was made for: scale anew (s is never negative, so
      // its bits compare as integers).
      const uint32_t top = __vmaxu2(__vmaxu2(vm[0], vm[1]), __vmaxu2(vm[2], vm[3])) & s_mask;
      if (__any_sync(0xffffffffu, __vmaxu2(top, s_most) != s_most)) {
        const uint32_t bits = max(__reduce_max_sync(0xffffffffu, max(top & 0xFFFFu, top >> 16)) >> 10, 1u);
        if (s_most != 0u) {
          const float a = __uint_as_float((127u + max(s_most >> 26, 4u) - max(bits, 4u)) << 23);
#pragma unroll
          for (int j = 0; j < MB; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[j][i] *= a;
        }
        s_most = (((bits + 1) << 10) - 1) * 0x00010001u;
      }
    }
    // 2^-E: the largest s becomes 2^4 .. 2^5 (less where that would need more than 2^15)
    [[maybe_unused]] const uint32_t s_scale = 34u * kExponent - max(s_most & 0x7C007C00u, 4u * kExponent);
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      if constexpr (kF32) {
        l_sum[0] += t[hf][0] + t[hf][2];
        l_sum[1] += t[hf][1] + t[hf][3];
      } else {
        mma_f16(om, vm[2 * hf], kOnes, vm[2 * hf + 1], kOnes, pb[hf][0], pb[hf][1]);
      }
      uint32_t x[4];  // of two pieces: half word gq of tokens 2 tq, 2 tq + 1 and of those 8 on
      uint32_t b0, b1;
      [[maybe_unused]] uint32_t l0, l1;
      [[maybe_unused]] float undo[2];  // the powers of two that the products of heads 2 tq, 2 tq + 1 lack,
      [[maybe_unused]] float pm[2];    // and the sums of p m over the 16 tokens
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        if (i % 2 == 0) ldsm4_trans(x, st + kChunk + hf * kHalf * R + c_at[i / 2]);
        if (i % PG == 0 && kF32) {  // p s and p m of the group
          float x[4], hi[4], lo[4], m[2];
#pragma unroll
          for (int u = 0; u < 2; ++u)
            m[u] = fmaf(16.f, f16_lo(vpar[hf][u][i / PG]), f16_lo(vpar[hf][u][i / PG] >> 16));
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            pm[e] = fmaf(t[hf][2 + e], m[1], t[hf][e] * m[0]);
#pragma unroll
            for (int k = 4; k < 32; k <<= 1) pm[e] += __shfl_xor_sync(0xffffffffu, pm[e], k);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = t[hf][e] * f16_lo(vpar[hf][e / 2][i / PG]);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float most = fmaxf(x[e], x[e + 2]);
#pragma unroll
            for (int k = 4; k < 32; k <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, k));
            const uint32_t eb = max(__float_as_uint(most) >> 23, 20u);
            const float scale = __uint_as_float((260u - eb) << 23);  // the largest becomes 2^6 .. 2^7
            undo[e] = __uint_as_float((eb + 12u) << 23);             // with the codes' 2^-18
            split<-4>(x[e] * scale, hi[e], lo[e]);
            split<-4>(x[e + 2] * scale, hi[e + 2], lo[e + 2]);
          }
          b0 = movm_trans(pack_f16x2(hi[0], hi[1]));
          b1 = movm_trans(pack_f16x2(hi[2], hi[3]));
          l0 = movm_trans(pack_f16x2(lo[0], lo[1]));
          l1 = movm_trans(pack_f16x2(lo[2], lo[3]));
        } else if (i % PG == 0) {
          const int from = s_lane + i / PG * 8;
          b0 = mul_f16x2(pb[hf][0], mul_f16x2(__shfl_sync(0xffffffffu, vm[2 * hf], from), s_scale));
          b1 = mul_f16x2(pb[hf][1], mul_f16x2(__shfl_sync(0xffffffffu, vm[2 * hf + 1], from), s_scale));
        }
        const uint32_t x0 = i % 2 == 0 ? x[0] : x[2], x1 = i % 2 == 0 ? x[1] : x[3];
        const uint32_t y0 = __byte_perm(x0, 0, 0x2301), y1 = __byte_perm(x1, 0, 0x2301);
        if constexpr (kF32) {
          float d[4][4] = {};
          mma_f16(d[0], raw_hi(x0), raw_hi(y0), raw_hi(x1), raw_hi(y1), b0, b1);
          mma_f16(d[1], raw_hi(x0), raw_hi(y0), raw_hi(x1), raw_hi(y1), l0, l1);
          mma_f16(d[2], raw_lo(x0), raw_lo(y0), raw_lo(x1), raw_lo(y1), b0, b1);
          mma_f16(d[3], raw_lo(x0), raw_lo(y0), raw_lo(x1), raw_lo(y1), l0, l1);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            o[2 * i][e] += fmaf(d[0][e] + d[1][e], undo[e & 1], pm[e & 1]);
            o[2 * i + 1][e] += fmaf(d[2][e] + d[3][e], undo[e & 1] * 16.f, pm[e & 1]);
          }
        } else {
          mma_f16(o[2 * i], raw_hi(x0), raw_hi(y0), raw_hi(x1), raw_hi(y1), b0, b1);
          mma_f16(o[2 * i + 1], raw_lo(x0), raw_lo(y0), raw_lo(x1), raw_lo(y1), b0, b1);
        }
      }
    }
    uint32_t b = 0, share = 0;
    if (flags & kLast) {
      b = lds32(md);
      share = lds32(md + 8);
    }
    __syncwarp();
    if (lane == 0) bar_arrive(empty(s));

    if (!kF32 && (flags & (kLast | kYield | kSettle))) {
      // the second term joins the first, in the first's powers of two
      const float hi = __uint_as_float((127u - 18 + 19 - max(s_most >> 26, 4u)) << 23), lo = hi * 0.0625f;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        float add[2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
          add[e] = fmaf(16.f, __shfl_sync(0xffffffffu, om[e], s_lane + 8 * g),
                        __shfl_sync(0xffffffffu, om[e], s_lane + 8 * g + 4));
#pragma unroll
        for (int j = g * 2 * PG; j < (g + 1) * 2 * PG; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[j][i] = fmaf(add[i & 1], (j & 1) ? lo : hi, o[j][i]);
      }
      om[0] = om[1] = 0.f;
    }
    if (flags & (kLast | kYield)) {
      float l[2] = {om[2], om[3]};  // the softmax sums
      if constexpr (kF32) {
#pragma unroll
        for (int k = 4; k < 32; k <<= 1)
#pragma unroll
          for (int e = 0; e < 2; ++e) l_sum[e] += __shfl_xor_sync(0xffffffffu, l_sum[e], k);
        l[0] = l_sum[0];
        l[1] = l_sum[1];
      } else {
        // the powers of two undone
        const float hi = __uint_as_float((127u + 18 - 19 + max(s_most >> 26, 4u)) << 23), lo = hi * 16.f;
#pragma unroll
        for (int j = 0; j < MB; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[j][i] *= (j & 1) ? lo : hi;
      }
      if (flags & kYield) {
        // hand this group's part over: once the previous one has been taken
        if (!wait(taken(), hand_phase ^ 1)) break;
        hand_phase ^= 1;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int g = 2 * tq + e;
          if (g < G) {
            float* dst = reinterpret_cast<float*>(smem + p.off_hand) + (h * G + g) * (HD + 4);
#pragma unroll
            for (int j = 0; j < MB; j += 2)
              *reinterpret_cast<float4*>(dst + j * 16 + gq * 4) =
                  make_float4(o[j][e], o[j][2 + e], o[j + 1][e], o[j + 1][2 + e]);
            if (gq == 0) *reinterpret_cast<float2*>(dst + HD) = make_float2(m[e], l[e]);
          }
        }
        __syncwarp();
        if (lane == 0) bar_arrive(handed());
        continue;
      }
      if (!(flags & kSolo)) {
        // add the other group's part
        if (!wait(handed(), hand_phase)) break;
        hand_phase ^= 1;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int g = 2 * tq + e;
          if (g < G) {
            const float* src = reinterpret_cast<const float*>(smem + p.off_hand) + (h * G + g) * (HD + 4);
            const float2 ml = *reinterpret_cast<const float2*>(src + HD);
            // a part without tokens (bad pages) has sum 0 and no say in the reference
            const float mm = ml.y == 0.f ? m[e] : l[e] == 0.f ? ml.x : fmaxf(m[e], ml.x);
            const float wa = l[e] == 0.f ? 0.f : ex2_approx(m[e] - mm), wb = ml.y == 0.f ? 0.f : ex2_approx(ml.x - mm);
            m[e] = mm;
            l[e] = l[e] * wa + ml.y * wb;
#pragma unroll
            for (int j = 0; j < MB; j += 2) {
              const float4 v = *reinterpret_cast<const float4*>(src + j * 16 + gq * 4);
              o[j][e] = o[j][e] * wa + v.x * wb;
              o[j][2 + e] = o[j][2 + e] * wa + v.y * wb;
              o[j + 1][e] = o[j + 1][e] * wa + v.z * wb;
              o[j + 1][2 + e] = o[j + 1][2 + e] * wa + v.w * wb;
            }
          }
        }
        __syncwarp();
        if (lane == 0) bar_arrive(taken());
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int g = 2 * tq + e;
        if (g < G) {
          const float inv = l[e] > 0.f ? 1.f / l[e] : 0.f;
          const int hq = h * G + g;
          if (flags & kWhole) {
            char* dst = p.k.out + (static_cast<int64_t>(b) * p.k.Hq + hq) * HD * sizeof(T);
#pragma unroll
            for (int j = 0; j < MB; j += 2) {
              char* at = dst + (j * 16 + gq * 4) * sizeof(T);
              if constexpr (kF32)
                *reinterpret_cast<float4*>(at) =
                    make_float4(o[j][e] * inv, o[j][2 + e] * inv, o[j + 1][e] * inv, o[j + 1][2 + e] * inv);
              else
                *reinterpret_cast<uint2*>(at) = make_uint2(pack_bf16x2(o[j][e] * inv, o[j][2 + e] * inv),
                                                           pack_bf16x2(o[j + 1][e] * inv, o[j + 1][2 + e] * inv));
            }
          } else {
            // a partial result: for the merge kernel, or (generic addresses) for the cluster
            const int64_t part = (static_cast<int64_t>(share) + b) * p.k.Hq + hq;
            float* dst = p.k.o_part + part * HD;
            float* lse = p.k.lse_part + part;
            if (p.cluster) {
              dst = reinterpret_cast<float*>(smem + p.off_hand) + hq * (HD + 4);
              lse = dst + HD;
            }
#pragma unroll
            for (int j = 0; j < MB; j += 2)
              *reinterpret_cast<float4*>(dst + j * 16 + gq * 4) =
                  make_float4(o[j][e] * inv, o[j][2 + e] * inv, o[j + 1][e] * inv, o[j + 1][2 + e] * inv);
            if (gq == 0) *lse = partial_lse(m[e], l[e]);
          }
        }
      }
      __syncwarp();
    }
  }
}

// ---------------------------------------------------------------------------
// producer warp
// ---------------------------------------------------------------------------
// The chunk prefix sums of up to kInlinePlanMax requests, by one warp into
// shared memory: each lane sums a run of consecutive requests, so one round
// trip of loads and one warp scan.  `first` (the warp of share 0) also does the
// plan's side work, as plan_in_cta.
PA_DEVINL int plan_in_warp(const KParams& k, int32_t* cs_s, bool first, int lane) {
  const int cap = static_cast<int>(min(static_cast<int64_t>(k.max_ctx), static_cast<int64_t>(k.maxp) << k.log2P));
  const int per = (k.B + 31) / 32;
  const int b0 = min(k.B, lane * per), b1 = min(k.B, b0 + per);
  int sum = 0;
#pragma unroll 8
  for (int b = b0; b < b1; ++b) {
    const int L = k.ctx[b];
    int cnt = 0;
    if (L >= 1 && L <= cap) {
      cnt = (L + kTok - 1) / kTok;
    } else if (first) {
      // length 0 is a padding row: nothing is read, stored or written for it
      if (L != 0) raise_flag(k.err, PA_DEVERR_BAD_LENGTH);
      if (k.k_new != nullptr && k.slot_out) k.slot_out[b] = -1;
    }
    cs_s[b + 1] = cnt;
    sum += cnt;
  }
  int x = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  int run = x - sum;
  for (int b = b0; b < b1; ++b) {
    run += cs_s[b + 1];
    cs_s[b + 1] = run;
  }
  if (lane == 0) cs_s[0] = 0;
  __syncwarp();
  return __shfl_sync(0xffffffffu, x, 31);
}

// Fills the ring with the chunks of this CTA's share.
PA_DEVINL void produce(const Q4Params& p, unsigned char* smem, uint64_t* full, uint64_t* empty, int4* meta,
                       volatile int* abort_flag, int lane) {
  const KParams& k = p.k;
  const uint64_t pol = l2_policy_evict_first();
  const int32_t* cs;
  int NC;
  if (k.inline_plan) {
    int32_t* cs_s = reinterpret_cast<int32_t*>(smem + k.off_cs);
    NC = plan_in_warp(k, cs_s, blockIdx.x == 0, lane);
    cs = cs_s;
  } else {
    pdl_wait();  // the plan kernel's chunk sums are complete
    cs = k.cs;
    NC = cs[k.B];
  }
  const int c = blockIdx.x;
  // its share: of its cluster's request, or of the batch
  int b, x0, x1;
  if (p.cluster) {
    b = c / p.cluster;
    const int part = c - b * p.cluster, count = cs[b + 1] - cs[b];
    x0 = cs[b] + part * count / p.cluster;
    x1 = cs[b] + (part + 1) * count / p.cluster;
  } else {
    x0 = static_cast<int>((static_cast<int64_t>(c) * NC) / k.n_ctas);
    x1 = static_cast<int>((static_cast<int64_t>(c + 1) * NC) / k.n_ctas);
    b = x0 < x1 ? first_request(cs, k.B, x0) : 0;
  }
  const uint32_t rb = static_cast<uint32_t>(k.row_bytes), q_bytes = p.stage_bytes - 2 * k.chunk_bytes;
  int issued = 0;
  Ring ring;
  bool aborted = false;
  for (int xg = x0; xg < x1 && !aborted; xg += 32) {
    // a lane looks up one of the next 32 chunks, then issues its copies in turn
    const int nvalid = min(32, x1 - xg);
    const int x = xg + lane;
    int my_b = b, n[2] = {0, 0}, new_slot = -1;
    uint32_t flags = 0;
    bool ends = false;
    long long off[2] = {0, 0};
    if (lane < nvalid) {
      while (my_b < k.B - 1 && cs[my_b + 1] <= x) ++my_b;
      const int cb0 = cs[my_b], cb1 = cs[my_b + 1];
      const int t0 = (x - cb0) * kTok;
      const int left = k.ctx[my_b] - t0;
      const int32_t* bt = k.bt + static_cast<int64_t>(my_b) * k.maxp;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int th = t0 + hf * kHalf, nh = min(kHalf, left - hf * kHalf);
        if (nh <= 0) continue;
        const int page = bt[th >> k.log2P];
        if (page < 0 || page >= k.num_pages) {
          raise_flag(k.err, PA_DEVERR_BAD_PAGE);
          continue;
        }
        const long long slot0 = (static_cast<long long>(page) << k.log2P) + (th & (k.P - 1));
        off[hf] = slot0 * k.row_bytes;
        n[hf] = nh;
        if (k.k_new != nullptr && th + nh == t0 + left) new_slot = static_cast<int>(slot0) + nh - 1;  // the last token
      }
      ends = x == cb1 - 1;
      const int xa = max(x0, cb0), xb = min(x1, cb1);  // the request's chunks in this share
      flags = (x < xa + p.groups ? kFirst : 0u) | (x == xb - 1 ? kLast : 0u) |
              (p.groups == 2 && x == xb - 2 ? kYield : 0u) | (p.groups == 1 || xb - xa == 1 ? kSolo : 0u) |
              (cb0 >= x0 && cb1 <= x1 && p.cluster <= 1 ? kWhole : 0u) |
              (n[0] != kHalf || n[1] != kHalf ? kRagged : 0u) | (new_slot >= 0 ? kNew : 0u) |
              ((x - xa) / p.groups % kSettleChunks == kSettleChunks - 1 ? kSettle : 0u);
    }
    b = __shfl_sync(0xffffffffu, my_b, nvalid - 1);
    for (int u = 0; u < nvalid; ++u, ring.next(p.stages)) {
      int ok = 1;
      if (lane == u) {
        const int s = ring.s;
        if (!mbar_wait_bounded(&empty[s], ring.phase ^ 1, abort_flag, k.err)) {
          ok = 0;
        } else {
          meta[s] = make_int4(my_b, n[0] | n[1] << 8 | static_cast<int>(flags), c, new_slot);
          // the new token's row is quantised by the consumers
          int rows0 = n[0], rows1 = n[1];
          if (new_slot >= 0) {
            if (rows1) --rows1;
            else --rows0;
          }
          const uint32_t qb = (flags & kFirst) ? q_bytes : 0u;
          unsigned char* dst = smem + static_cast<size_t>(s) * p.stage_bytes;
          mbar_arrive_expect_tx(&full[s], 2 * rb * static_cast<uint32_t>(rows0 + rows1) + qb);
          if (rows0 == kHalf && off[1] == off[0] + kHalf * static_cast<long long>(rb)) {  // one run
            rows0 += rows1;
            rows1 = 0;
          }
          if (qb) bulk_g2s(dst + 2 * k.chunk_bytes, k.q + static_cast<int64_t>(my_b) * q_bytes, qb, &full[s]);
          if (rows0 > 0) {
            bulk_g2s_hint(dst, k.k_cache + off[0], rows0 * rb, &full[s], pol);
            bulk_g2s_hint(dst + k.chunk_bytes, k.v_cache + off[0], rows0 * rb, &full[s], pol);
          }
          if (rows1 > 0) {
            bulk_g2s_hint(dst + kHalf * rb, k.k_cache + off[1], rows1 * rb, &full[s], pol);
            bulk_g2s_hint(dst + k.chunk_bytes + kHalf * rb, k.v_cache + off[1], rows1 * rb, &full[s], pol);
          }
          if (k.k_new != nullptr && ends && k.slot_out) k.slot_out[my_b] = new_slot;
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, u);
      if (!ok) {
        aborted = true;
        break;
      }
      ++issued;
    }
  }
  if (lane == 0) {
    if (aborted) {
      // Copies already issued may still be landing: wait for them (time only).
      for (int it = max(0, issued - p.stages); it < issued; ++it)
        drain_wait(&full[it % p.stages], (it / p.stages) & 1);
    } else {
      for (int g = 0; g < p.groups; ++g, ring.next(p.stages)) {  // one end for each group
        if (!mbar_wait_bounded(&empty[ring.s], ring.phase ^ 1, abort_flag, k.err)) break;
        meta[ring.s] = make_int4(0, static_cast<int>(kEnd), 0, -1);
        mbar_arrive(&full[ring.s]);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// The partial results of a cluster's request, which its CTAs left in their shared
// memory (off_hand, with the log2-sum-exp behind the outputs; -infinity where a
// CTA had no chunk): a warp takes a q-head and adds them in the order of the CTAs.
// ---------------------------------------------------------------------------
PA_DEVINL void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
PA_DEVINL uint32_t peer_addr(uint32_t a, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  return r;
}

template <typename T, int HD>
PA_DEVINL void cluster_merge(const Q4Params& p, unsigned char* smem, int warp, int lane) {
  constexpr int EL = HD / 32;
  cluster_sync();  // every part is in its place
  const int b = blockIdx.x / p.cluster, rank = blockIdx.x - b * p.cluster;
  const int32_t* cs = reinterpret_cast<const int32_t*>(smem + p.k.off_cs);
  if (cs[b] < cs[b + 1]) {  // (a padding row keeps its output)
    const int nw = blockDim.x / 32;
    for (int hq = rank * nw + warp; hq < p.k.Hq; hq += p.cluster * nw) {
      const uint32_t at = smem_u32(smem) + p.off_hand + hq * (HD + 4) * 4;
      float lse = -INFINITY;  // lane r: CTA r's
      if (lane < p.cluster)
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(lse) : "r"(peer_addr(at + HD * 4, lane)));
      float v[kMaxCluster][EL];
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        if (r >= p.cluster) break;
        const uint32_t src = peer_addr(at + lane * EL * 4, r);
        if constexpr (EL == 4)
          asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(v[r][0]), "=f"(v[r][1]), "=f"(v[r][2]), "=f"(v[r][3])
                       : "r"(src));
        else
          asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v[r][0]), "=f"(v[r][1]) : "r"(src));
      }
      float top = lse;
#pragma unroll
      for (int o = 4; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float w = lse == -INFINITY ? 0.f : ex2_approx(lse - top);
      float sum = w;
#pragma unroll
      for (int o = 4; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      sum = __shfl_sync(0xffffffffu, sum, 0);
      const float inv = sum > 0.f ? 1.f / sum : 0.f;
      float acc[EL] = {};
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        if (r >= p.cluster) break;
        const float wr = __shfl_sync(0xffffffffu, w, r);
        if (wr != 0.f)  // (a CTA without a chunk left nothing)
#pragma unroll
          for (int e = 0; e < EL; ++e) acc[e] = fmaf(wr, v[r][e], acc[e]);
      }
      T* dst = reinterpret_cast<T*>(p.k.out) + (static_cast<int64_t>(b) * p.k.Hq + hq) * HD + lane * EL;
#pragma unroll
      for (int e = 0; e < EL; e += 2) {
        if constexpr (sizeof(T) == 4)
          *reinterpret_cast<float2*>(dst + e) = make_float2(acc[e] * inv, acc[e + 1] * inv);
        else
          *reinterpret_cast<uint32_t*>(dst + e) = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
      }
    }
  }
  cluster_sync();  // no CTA leaves while its part is read
}

// bf16: two groups of one consumer warp per kv-head, which take the chunks in
// turn from one ring, and the producer; fp32: one group.  NG: the groups of a
// head's row, HKV: kv-heads (a row's layout in the instructions: 27 address
// additions a chunk less).
template <typename T, int HD, int NG, int HKV>
__global__ void __launch_bounds__(sizeof(T) == 2 ? 17 * 32 : 9 * 32, 1)
    decode_q4_kernel(const Q4Params p) {
  extern __shared__ __align__(128) unsigned char smem[];
  const KParams& k = p.k;
  const int NW = k.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + k.off_bar);
  uint64_t* empty = full + kMaxStages;
  uint64_t* handed = empty + kMaxStages;  // [8] per kv-head: a part is in its place
  uint64_t* taken = handed + 8;           // [8] it has been added
  int4* meta = reinterpret_cast<int4*>(smem + k.off_meta);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + k.off_abort);
  if (p.cluster > 1)
    for (int hq = threadIdx.x; hq < k.Hq; hq += blockDim.x)
      *reinterpret_cast<float*>(smem + p.off_hand + (hq * (HD + 4) + HD) * 4) = -INFINITY;
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], NW);
    }
    for (int h = 0; h < NW; ++h) {
      mbar_init(&handed[h], 1);
      mbar_init(&taken[h], 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  cta_sync();
  pdl_trigger();  // the merge kernel may start launching; it waits for this grid

  if (warp == NW * p.groups) {
    produce(p, smem, full, empty, meta, abort_flag, lane);
  } else {
    const int group = warp >= NW;
    consume<T, HD, NG, HKV>(p, smem, warp - group * NW, group);
  }
  __syncwarp();
  if (p.cluster > 1) cluster_merge<T, HD>(p, smem, warp, lane);
}

struct Fns {
  const void* main;
  const void* merge;
};

template <typename T, int HD, int HKV>
const void* main_fn(int gs) {
  if constexpr (HD == 128)
    if (gs == 32) return reinterpret_cast<const void*>(decode_q4_kernel<T, HD, 4, HKV>);
  return HD == 2 * gs ? reinterpret_cast<const void*>(decode_q4_kernel<T, HD, 2, HKV>)
                      : reinterpret_cast<const void*>(decode_q4_kernel<T, HD, 1, HKV>);
}

template <typename T, int HD>
Fns fns_for(int hkv, int gs) {
  const void* merge = reinterpret_cast<const void*>(decode_merge_kernel<T, HD>);
  switch (hkv) {
    case 1: return {main_fn<T, HD, 1>(gs), merge};
    case 2: return {main_fn<T, HD, 2>(gs), merge};
    case 4: return {main_fn<T, HD, 4>(gs), merge};
    default: return {main_fn<T, HD, 8>(gs), merge};
  }
}

Fns get_fns(const pa_cache_desc& d, int gs) {
  const int hkv = d.num_kv_heads;
  if (d.dtype == PA_BF16)
    return d.head_dim == 128 ? fns_for<__nv_bfloat16, 128>(hkv, gs) : fns_for<__nv_bfloat16, 64>(hkv, gs);
  return d.head_dim == 128 ? fns_for<float, 128>(hkv, gs) : fns_for<float, 64>(hkv, gs);
}

// Bytes of a ring stage: a chunk's rows of K and V, and a request's queries.
size_t q4_stage_bytes(const pa_cache_desc& d, const DecodePlan& pl) {
  return 2 * static_cast<size_t>(pl.chunk_bytes) +
         static_cast<size_t>(d.num_q_heads) * d.head_dim * elem_bytes(d.dtype);
}

int q4_groups(const pa_cache_desc& d) { return d.dtype == PA_BF16 ? 2 : 1; }

}  // namespace

cudaError_t plan_decode_q4(const pa_cache_desc& d, int gs, int batch, int max_ctx, int max_ctas, DecodePlan* out) {
  DeviceInfo di;
  cudaError_t e = current_device_info(&di);
  if (e != cudaSuccess) return e;
  DecodePlan pl;
  pl.nw = d.num_kv_heads * q4_groups(d);  // consumer warps
  pl.tokens_per_chunk = kTok;
  pl.row_pitch = q4_row_bytes(d, gs);
  pl.chunk_bytes = pl.tokens_per_chunk * pl.row_pitch;
  // behind the ring: barriers, chunk descriptors, the batch's prefix sums, and
  // the part that is handed over
  size_t off = 0;
  auto place = [&](size_t bytes) {
    const size_t at = off;
    off = align_up(off + bytes, 16);
    return static_cast<uint32_t>(at);
  };
  pl.off_bar = place((2 * kMaxStages + 16) * sizeof(uint64_t));
  pl.off_meta = place(kMaxStages * 16);
  pl.off_abort = place(16);
  pl.off_cs = place(static_cast<size_t>(kInlinePlanMax + 1 + 32) * 4);
  pl.off_ml = place(static_cast<size_t>(d.num_q_heads) * (d.head_dim + 4) * 4);
  // The ring takes what is left of a CTA's share of the SM's shared memory with
  // 8 kv-heads on an SM: four or more chunks (of fp32, with many q-heads, two).
  const size_t fixed = align_up(off, 128), stage = q4_stage_bytes(d, pl);
  const size_t share = static_cast<size_t>(di.max_smem_optin) * d.num_kv_heads / 8 - 1024;
  const size_t room = share > fixed ? (share - fixed) / stage : 0;
  pl.stages = static_cast<int>(std::min<size_t>(kMaxStages, std::max<size_t>(2, room)));
  const uint32_t ring = static_cast<uint32_t>(pl.stages * stage);  // the ring comes first
  for (uint32_t* o : {&pl.off_bar, &pl.off_meta, &pl.off_abort, &pl.off_cs, &pl.off_ml})
    *o += ring;
  pl.smem_bytes = ring + fixed;
  if (pl.smem_bytes > static_cast<size_t>(di.max_smem_optin)) return cudaErrorInvalidValue;
  int occ = 0;
  e = ctas_per_sm(di, get_fns(d, gs).main, (pl.nw + 1) * 32, pl.smem_bytes, &occ);
  if (e != cudaSuccess) return e;
  const int T = pl.tokens_per_chunk;
  const int64_t chunks_upper = static_cast<int64_t>(batch) * ((static_cast<int64_t>(max_ctx) + T - 1) / T);
  int64_t n = static_cast<int64_t>(occ) * di.sm_count;
  if (max_ctas > 0) n = std::min<int64_t>(n, max_ctas);
  // Short requests that fit the GPU at once: a CTA or a cluster each and no merge
  // kernel, 2 to 4 us of such a call; against them the GPU's other SMs.  With 32
  // q-heads over 8 of 128 dims, groups of 32, in us (the even split), bf16: 16
  // requests of 300-1000 tokens by clusters of 6 14.9 (16.5), 37 of 64-512 by 3 14.6
  // (15.9), 64 of 100-512 by 2 16.9 (18.3), 100 of 64-256 by one CTA each 15.8 (19.3),
  // 4 of 5-64 8.1 (8.8).  Longer parts: 64 of 300-2000 by 2 36.9 (28.3).  Too few: 2 of
  // 301-905 by 8 12.8 (11.2), 4 of 100-256 by one 13.1 (9.3).  fp32, the same: 23.4
  // (20.6), 23.9 (19.9), 29.7 (25.1), 28.6 (24.7), 10.5 (10.2); at half the length, 16
  // over 8 heads of 64 dims: 16 of 300-1000 by 6 13.8 (14.6), 64 of 100-512 by 2 16.4
  // (16.6), 152 of 64-256 by one 17.0 (20.8), 4 of 5-64 7.1 (8.1); 64 of 300-1000 by 2
  // 26.3 (21.9).
  if (batch >= 1 && batch <= kInlinePlanMax && n >= batch) {
    const int64_t work = static_cast<int64_t>(max_ctx) * d.head_dim * (d.dtype == PA_BF16 ? 1 : 2);
    const int64_t most = std::min<int64_t>({kMaxCluster, n / batch, chunks_upper / batch});
    for (int c = work <= kAloneTokens * 128 ? 1 : static_cast<int>(most); c >= 1; --c) {
      const bool fills = 5 * static_cast<int64_t>(batch) * c >= 2 * di.sm_count;
      if (work > (fills ? c * kPartTokens : c == 1 ? kAloneTokens : 0) * 128) continue;
      int fit = batch;
      if (c > 1) {
        e = ctas_per_sm(di, get_fns(d, gs).main, (pl.nw + 1) * 32, pl.smem_bytes, &fit, c);
        if (e != cudaSuccess) return e;
      }
      if (fit < batch) continue;
      pl.cluster = c;
      break;
    }
  }
  n = std::min<int64_t>(n, std::max<int64_t>(1, chunks_upper));
  pl.n_ctas = static_cast<int>(std::max<int64_t>(1, n));
  decode_workspace_layout(d, batch, &pl);  // (the same for both forms: it grows with the bounds)
  if (pl.cluster) pl.n_ctas = batch * pl.cluster;
  *out = pl;
  return cudaSuccess;
}

cudaError_t launch_decode_q4(const pa_cache_desc& d, int gs, const DecodePlan& pl, const DecodeArgs& a,
                             cudaStream_t s) {
  const Fns f = get_fns(d, gs);
  Q4Params p{};
  p.k = decode_params(d, pl, a, q4_row_bytes(d, gs));
  p.stages = pl.stages;
  p.stage_bytes = static_cast<int32_t>(q4_stage_bytes(d, pl));
  p.codes = q4_codes_bytes(d);
  p.pars = p.k.row_bytes - p.codes;
  while ((1 << p.log2gs) < gs) ++p.log2gs;
  p.groups = q4_groups(d);
  p.cluster = pl.cluster;
  p.off_hand = pl.off_ml;
  void* args[] = {&p};
  return launch_decode_kernels(f.main, f.merge, pl, p.k, args, s);
}

}  // namespace pa
