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
  return g;
}

// The code of one clamped value: rint((x - c) / s) - 16 within 0..15.
PA_DEVINL uint32_t q4_code(float x, const Q4Group& g) {
  float t = __fmul_rn(__fsub_rn(x, g.c), g.r);
  t = fminf(fmaxf(t, 16.f), 31.f);
  // adding 1.5 * 2^23 rounds to an integer (half to even) in the low bits
  return __float_as_uint(__fadd_rn(t, 12582912.f)) & 15u;
}

// Four consecutive dims' codes in their 16 bits.
PA_DEVINL uint32_t q4_pack4(uint32_t u0, uint32_t u1, uint32_t u2, uint32_t u3) {
  return (u0 << 6) | (u2 << 2) | (u3 << 10) | ((u1 & 3u) << 14) | (u1 >> 2);
}

PA_DEVINL uint32_t q4_encode4(const float (&x)[4], const Q4Group& g) {
  return q4_pack4(q4_code(x[0], g), q4_code(x[1], g), q4_code(x[2], g), q4_code(x[3], g));
}

PA_DEVINL float q4_clamp(float x) { return fminf(fmaxf(x, -kQ4Max), kQ4Max); }
PA_DEVINL bool q4_bad(float x) { return !(fabsf(x) <= FLT_MAX); }

// Eight elements of the storage type as fp32.
template <typename T>
PA_DEVINL void q4_load8(const char* p, float (&x)[8]) {
  if constexpr (sizeof(T) == 2) {
    const uint4 w = ldg16(p);
    const float2 a = bf16x2_to_float2(w.x), b = bf16x2_to_float2(w.y), c = bf16x2_to_float2(w.z),
                 d = bf16x2_to_float2(w.w);
    x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
    x[4] = c.x; x[5] = c.y; x[6] = d.x; x[7] = d.y;
  } else {
    const uint4 w = ldg16(p), v = ldg16(p + 16);
    x[0] = __uint_as_float(w.x); x[1] = __uint_as_float(w.y); x[2] = __uint_as_float(w.z); x[3] = __uint_as_float(w.w);
    x[4] = __uint_as_float(v.x); x[5] = __uint_as_float(v.y); x[6] = __uint_as_float(v.z); x[7] = __uint_as_float(v.w);
  }
}

// Eight consecutive dims of a group spread over `lanes` (a power of two)
// neighbouring lanes, all 32 lanes taking part: the word of codes, and the
// group's parameters.
PA_DEVINL uint32_t q4_quantise8(float (&x)[8], int lanes, uint32_t& params) {
  bool bad = false;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    bad |= q4_bad(x[e]);
    x[e] = q4_clamp(x[e]);
  }
  float mn = x[0], mx = x[0];
#pragma unroll
  for (int e = 1; e < 8; ++e) {
    mn = fminf(mn, x[e]);
    mx = fmaxf(mx, x[e]);
  }
#pragma unroll
  for (int m = 1; m < lanes; m <<= 1) {
    mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, m));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, m));
    bad |= __shfl_xor_sync(0xffffffffu, static_cast<int>(bad), m) != 0;
  }
  const Q4Group g = q4_group(mn, mx, bad);
  params = g.word;
  const float a[4] = {x[0], x[1], x[2], x[3]}, b[4] = {x[4], x[5], x[6], x[7]};
  return q4_encode4(a, g) | (q4_encode4(b, g) << 16);
}

// The value of one code of a group (one fp32 rounding: s * (16 + u) is exact).
PA_DEVINL float q4_value(uint32_t u, float s, float c) { return fmaf(s, static_cast<float>(16u + u), c); }

PA_DEVINL void q4_decode4(uint32_t h, float s, float c, float (&x)[4]) {
  x[0] = q4_value((h >> 6) & 15u, s, c);
  x[1] = q4_value(((h >> 14) & 3u) | ((h & 3u) << 2), s, c);
  x[2] = q4_value((h >> 2) & 15u, s, c);
  x[3] = q4_value((h >> 10) & 15u, s, c);
}

PA_DEVINL float2 q4_sc(uint32_t word) {
  return make_float2(__half2float(__ushort_as_half(static_cast<uint16_t>(word & 0xFFFFu))),
                     __half2float(__ushort_as_half(static_cast<uint16_t>(word >> 16))));
}

}  // namespace pa
