// The 4-bit cache row: layout, quantisation and decoding (sm_103a).
//
// One token's row of K (or V) holds, for all kv-heads,
//   codes   Hkv * HD / 2 bytes: head h's codes at h * HD / 2
//   params  Hkv * HD / GS words, padded to 16 bytes: group g of head h at word
//           h * (HD / GS) + g, float16 s in its low and c in its high half
// and a code u (0..15) of the group stands for s * (16 + u) + c.
//
// Why 16 + u: with u in bits 6-9 of a half word, the float16 whose bits are
// 0x4C00 | u << 6 is exactly 16 + u, so a code becomes a float16 by one
// mask-or, and its value by one fused multiply-add with (s, c).
//
// 16 bits of codes hold four consecutive dims, each four bits wide:
//   dim 0 in bits 6-9      dim 2 in bits 2-5    (4 left of it: bits 6-9)
//   dim 1 in bits 14, 15, 0, 1 (low to high)    dim 3 in bits 10-13
// With the two bytes swapped, dims 1 and 3 take the places of dims 0 and 2.
//
// Swizzle: within each part, inside blocks of up to 128 bytes, the 16-byte
// piece j of slot t's row lies at piece j ^ (t mod pieces).  Rows are copied
// to shared memory as they are; rows of one head in neighbouring tokens would
// otherwise start in the same banks (a row is often a multiple of 128 bytes).
#pragma once

#include <cuda_fp16.h>
#include <float.h>

#include "pa_common.cuh"

namespace pa {

constexpr float kQ4Max = 16384.f;             // larger magnitudes are clamped (c = min - 16 s stays a float16)
constexpr float kQ4Fifteenth = 1.0f / 15.0f;  // the fp32 number nearest to 1/15

// Byte offset of byte o of a swizzled part of `size` bytes (a power of two
// >= 16), in the row of a slot whose low bits are t.
PA_DEVINL uint32_t q4_swz(uint32_t o, uint32_t size, uint32_t t) {
  const uint32_t mask = min(size >> 4, 8u) - 1;  // pieces - 1
  return o ^ ((t & mask) << 4);
}

struct Q4Group {  // a group's parameters, as stored and as fp32
  uint32_t word;  // s | c << 16
  float c, r;     // r = 1 / s, or 0
  bool clamp;     // (x - c) / s may round beyond 16..31
};

// Parameters of a group with minimum mn and maximum mx (clamped values), or of
// a group that holds a NaN or an infinity (bad: s = 0, c = NaN).
PA_DEVINL Q4Group q4_group(float mn, float mx, bool bad) {
  const __half sh = __float2half_rn(__fmul_rn(__fsub_rn(mx, mn), kQ4Fifteenth));
  const float s = __half2float(sh);
  const __half ch = __float2half_rn(__fsub_rn(mn, 16.f * s));
  Q4Group g;
  g.word = bad ? 0x7E000000u
               : static_cast<uint32_t>(__half_as_ushort(sh)) | (static_cast<uint32_t>(__half_as_ushort(ch)) << 16);
  g.c = __half2float(ch);
  g.r = s > 0.f && !bad ? __frcp_rn(s) : 0.f;
  // With s a normal float16 (off by 2^-11 of itself at most) and |c| <= 512 s
  // (off by s / 4 at most), (x - c) / s lies within 16 - 0.26 .. 31 + 0.27 for
  // every x of the group, unless the range was clamped: no need to clamp.
  g.clamp = !(s >= 6.103515625e-5f && fabsf(g.c) <= 512.f * s && !bad && mn > -kQ4Max && mx < kQ4Max);
  return g;
}

// Two groups' parameters, each found by every second lane (lanes 2 i and 2 i + 1
// hold the same two ranges) and exchanged.
template <typename R>
PA_DEVINL void q4_group_pair(const R& a, const R& b, Q4Group& ga, Q4Group& gb) {
  const bool odd = threadIdx.x & 1;
  const Q4Group mine = R::select(odd, b, a).group();
  Q4Group other;
  other.word = __shfl_xor_sync(0xffffffffu, mine.word, 1);
  other.r = __shfl_xor_sync(0xffffffffu, mine.clamp ? -mine.r : mine.r, 1);  // (the flag in the sign)
  other.clamp = signbit(other.r);
  other.r = fabsf(other.r);
  other.c = __half2float(__ushort_as_half(static_cast<uint16_t>(other.word >> 16)));
  ga.word = odd ? other.word : mine.word;
  gb.word = odd ? mine.word : other.word;
  ga.r = odd ? other.r : mine.r;
  gb.r = odd ? mine.r : other.r;
  ga.c = odd ? other.c : mine.c;
  gb.c = odd ? mine.c : other.c;
  ga.clamp = odd ? other.clamp : mine.clamp;
  gb.clamp = odd ? mine.clamp : other.clamp;
}

// rint((x - c) / s), clamped to 16..31, in the low bits of an integer whose
// other bits are those of 1.5 * 2^23: adding that number rounds half to even.
// Values beyond +-kQ4Max need no clamp of their own: the group's range ends
// there, so they meet the ends of 16..31.
template <bool kClamp>
PA_DEVINL uint32_t q4_step(float x, const Q4Group& g) {
  const float t = __fmul_rn(__fsub_rn(x, g.c), g.r);
  return __float_as_uint(__fadd_rn(kClamp ? fminf(fmaxf(t, 16.f), 31.f) : t, 12582912.f));
}

// Eight dims' codes, four in each half of the word.  Dims 0, 2, 3 are shifted
// and added with their upper bits (each is 0x4B400010 + u), whose sum is taken
// off again; dim 1 is turned round the half word's end.
template <bool kClamp>
PA_DEVINL uint32_t q4_encode8_as(const float (&a)[4], const Q4Group& ga, const float (&b)[4], const Q4Group& gb) {
  constexpr uint32_t kBase = 0x4B400010u;
  constexpr uint32_t kBases = (kBase << 6) + (kBase << 2) + (kBase << 10) + (kBase << 22) + (kBase << 18) + (kBase << 26);
  const uint32_t u = (q4_step<kClamp>(a[0], ga) << 6) + (q4_step<kClamp>(a[2], ga) << 2) +
                     (q4_step<kClamp>(a[3], ga) << 10) + (q4_step<kClamp>(b[0], gb) << 22) +
                     (q4_step<kClamp>(b[2], gb) << 18) + (q4_step<kClamp>(b[3], gb) << 26) - kBases;
  const uint32_t v = (q4_step<kClamp>(a[1], ga) & 15u) | (q4_step<kClamp>(b[1], gb) << 16);  // (b's upper bits leave)
  return u | ((v << 14) & 0xC000C000u) | ((v >> 2) & 0x00030003u);
}

// All 32 lanes take part.
PA_DEVINL uint32_t q4_encode8(const float (&a)[4], const Q4Group& ga, const float (&b)[4], const Q4Group& gb) {
  return __any_sync(0xffffffffu, ga.clamp || gb.clamp) ? q4_encode8_as<true>(a, ga, b, gb)
                                                       : q4_encode8_as<false>(a, ga, b, gb);
}

PA_DEVINL bool q4_bad(float x) { return !(fabsf(x) <= FLT_MAX); }

// ----------------------------------------------------------------------------
// minimum and maximum of a group.  bf16: on packed pairs, as {min, -max}, with
// NaN passed on, so that one shuffle and one instruction take a step of the
// reduction; fp32: apart, with a flag for values that are not finite.
// ----------------------------------------------------------------------------
PA_DEVINL uint32_t min_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
PA_DEVINL uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

template <typename T>
struct Q4Range;

template <>
struct Q4Range<__nv_bfloat16> {
  uint32_t r;  // {min, -max}
  template <int N>
  PA_DEVINL void of_words(const uint32_t (&w)[N]) {
    uint32_t mn = w[0], mx = w[0];
#pragma unroll
    for (int i = 1; i < N; ++i) {
      mn = min_bf16x2(mn, w[i]);
      mx = max_bf16x2(mx, w[i]);
    }
    mx ^= 0x80008000u;
    r = min_bf16x2(__byte_perm(mn, mx, 0x5410), __byte_perm(mn, mx, 0x7632));
  }
  PA_DEVINL void join(const Q4Range& o) { r = min_bf16x2(r, o.r); }
  static PA_DEVINL Q4Range select(bool second, const Q4Range& b, const Q4Range& a) { return second ? b : a; }
  PA_DEVINL void reduce(int m) { r = min_bf16x2(r, __shfl_xor_sync(0xffffffffu, r, m)); }
  PA_DEVINL Q4Group group() const {
    const float mn = __uint_as_float(r << 16), mx = -__uint_as_float(r & 0xFFFF0000u);
    return q4_group(fminf(fmaxf(mn, -kQ4Max), kQ4Max), fmaxf(fminf(mx, kQ4Max), -kQ4Max), q4_bad(mn) || q4_bad(mx));
  }
};

template <>
struct Q4Range<float> {
  float mn, mx;
  int bad;
  template <int N>
  PA_DEVINL void of_words(const uint32_t (&w)[N]) {
    mn = INFINITY;
    mx = -INFINITY;
    bad = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float x = __uint_as_float(w[i]);
      bad |= q4_bad(x);
      mn = fminf(mn, x);
      mx = fmaxf(mx, x);
    }
  }
  PA_DEVINL void join(const Q4Range& o) {
    mn = fminf(mn, o.mn);
    mx = fmaxf(mx, o.mx);
    bad |= o.bad;
  }
  static PA_DEVINL Q4Range select(bool second, const Q4Range& b, const Q4Range& a) {
    Q4Range o;
    o.mn = second ? b.mn : a.mn;
    o.mx = second ? b.mx : a.mx;
    o.bad = second ? b.bad : a.bad;
    return o;
  }
  PA_DEVINL void reduce(int m) {
    Q4Range o;
    o.mn = __shfl_xor_sync(0xffffffffu, mn, m);
    o.mx = __shfl_xor_sync(0xffffffffu, mx, m);
    o.bad = __shfl_xor_sync(0xffffffffu, bad, m);
    join(o);
  }
  PA_DEVINL Q4Group group() const {
    return q4_group(fminf(fmaxf(mn, -kQ4Max), kQ4Max), fmaxf(fminf(mx, kQ4Max), -kQ4Max), bad != 0);
  }
};

// N words of the storage type as fp32 (bf16: two values a word).
template <typename T, int N, int M>
PA_DEVINL void q4_widen(const uint32_t (&w)[N], float (&x)[M]) {
  static_assert(N * 4 == M * static_cast<int>(sizeof(T)), "");
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (sizeof(T) == 2) {
      const float2 f = bf16x2_to_float2(w[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    } else {
      x[i] = __uint_as_float(w[i]);
    }
  }
}

// Words of eight elements of the storage type.
template <typename T>
constexpr int kQ4Words = 2 * sizeof(T);

template <typename T>
PA_DEVINL void q4_load8(const char* p, uint32_t (&w)[kQ4Words<T>]) {
#pragma unroll
  for (int i = 0; i < kQ4Words<T>; i += 4) {
    const uint4 v = ldg16(p + 4 * i);
    w[i] = v.x;
    w[i + 1] = v.y;
    w[i + 2] = v.z;
    w[i + 3] = v.w;
  }
}

// Eight consecutive dims of a group spread over `lanes` (a power of two, at
// least 4) neighbouring lanes, all 32 lanes taking part: the word of codes, and
// the group's parameters.
template <typename T>
PA_DEVINL uint32_t q4_quantise8(const uint32_t (&w)[kQ4Words<T>], int lanes, uint32_t& params) {
  Q4Range<T> range;
  range.of_words(w);
#pragma unroll
  for (int m = 1; m < lanes; m <<= 1) range.reduce(m);
  const Q4Group g = range.group();
  params = g.word;
  float x[8];
  q4_widen<T>(w, x);
  const float a[4] = {x[0], x[1], x[2], x[3]}, b[4] = {x[4], x[5], x[6], x[7]};
  return q4_encode8(a, g, b, g);
}

// The same of two rows (K and V).
template <typename T>
PA_DEVINL void q4_quantise8_pair(const uint32_t (&k)[kQ4Words<T>], const uint32_t (&v)[kQ4Words<T>], int lanes,
                                 uint32_t& k_codes, uint32_t& v_codes, uint32_t& k_params, uint32_t& v_params) {
  Q4Range<T> rk, rv;
  rk.of_words(k);
  rv.of_words(v);
#pragma unroll
  for (int m = 1; m < lanes; m <<= 1) {
    rk.reduce(m);
    rv.reduce(m);
  }
  Q4Group gk, gv;
  q4_group_pair(rk, rv, gk, gv);
  k_params = gk.word;
  v_params = gv.word;
  float x[8], y[8];
  q4_widen<T>(k, x);
  q4_widen<T>(v, y);
  const float a[4] = {x[0], x[1], x[2], x[3]}, b[4] = {x[4], x[5], x[6], x[7]};
  const float c[4] = {y[0], y[1], y[2], y[3]}, d[4] = {y[4], y[5], y[6], y[7]};
  if (__any_sync(0xffffffffu, gk.clamp || gv.clamp)) {
    k_codes = q4_encode8_as<true>(a, gk, b, gk);
    v_codes = q4_encode8_as<true>(c, gv, d, gv);
  } else {
    k_codes = q4_encode8_as<false>(a, gk, b, gk);
    v_codes = q4_encode8_as<false>(c, gv, d, gv);
  }
}

// The value of a code in bits 19-22, with one fp32 rounding (s * (16 + u) is
// exact): 16 + u is the fp32 number with u in bits 19-22 over 16's bits.
PA_DEVINL float q4_value(uint32_t code_at_19, float s, float c) {
  return fmaf(s, __uint_as_float((code_at_19 & 0x00780000u) | 0x41800000u), c);
}

// The eight values of a word of codes.
PA_DEVINL void q4_decode8(uint32_t w, float s, float c, float (&x)[8]) {
  const uint32_t lo = __byte_perm(w, 0, 0x1010), hi = __byte_perm(w, 0, 0x3232);  // a half twice: dim 1 in bits 14-17
  x[0] = q4_value(w << 13, s, c);
  x[1] = q4_value(lo << 5, s, c);
  x[2] = q4_value(w << 17, s, c);
  x[3] = q4_value(w << 9, s, c);
  x[4] = q4_value(w >> 3, s, c);
  x[5] = q4_value(hi << 5, s, c);
  x[6] = q4_value(w << 1, s, c);
  x[7] = q4_value(w >> 7, s, c);
}

PA_DEVINL float2 q4_sc(uint32_t word) {
  return make_float2(__half2float(__ushort_as_half(static_cast<uint16_t>(word & 0xFFFFu))),
                     __half2float(__ushort_as_half(static_cast<uint16_t>(word >> 16))));
}

}  // namespace pa
