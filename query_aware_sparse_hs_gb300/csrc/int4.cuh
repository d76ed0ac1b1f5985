// The 4-bit cache format: for every row and 32 channels a bf16 scale s, a bf16
// centre z and codes c of -8 .. 7, stored as c + 8, channel 2i in the low half of
// byte i.  A value is z + s c, in fp32.
//
// Of a group's values between lo and hi: z = (7 lo + 8 hi) / 15 rounded to bf16, so
// that c = -8 is lo and c = 7 is hi; s = max((hi - z) / 7, (z - lo) / 8) rounded up
// to bf16, so that every value has a code within s / 2 although z was rounded.  (A
// centre instead of a minimum: the codes' products are sums of both signs, which
// stay as small as the attention's result over long contexts, where sums of codes
// 0 .. 15 would have to cancel against the minimum's.)  bf16 for both: a centre of
// bf16 values of any size, and a group of equal values is held exactly.
#pragma once

#include "hs_common.cuh"

namespace hs {
namespace int4 {

// Two fp32 numbers at a time.
__device__ __forceinline__ float2 add_pair(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 mul_pair(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma_pair(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\tfma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

constexpr float kMost = 8.507059173023462e37f;        // 2^126: values beyond it are held as it
constexpr float kLeastScale = 1.2037062152420224e-35f;  // 2^-116: smaller ranges are held as their centre
constexpr float kRound = 12582920.0f;  // 1.5 2^23 + 8: c plus it is, as bits, round(c) + 8 more than 0x4b400000

__host__ __device__ constexpr int row_bytes(int head_dim) { return head_dim / 2; }
// scales and centres of a row, in 16-bit words
__host__ __device__ constexpr int record(int head_dim) { return 2 * (head_dim / kQuantGroup); }

// Least and largest of a group's values, and whether one is not a number (held as
// an infinite hi, which no other value leaves).
struct Range {
  float lo, hi;
  __device__ __forceinline__ void join(const Range& o) {
    lo = fminf(lo, o.lo);
    hi = fmaxf(hi, o.hi);
  }
  __device__ __forceinline__ void join_lane(int mask) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, mask));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, mask));
  }
};
__device__ __forceinline__ Range no_values() { return Range{INFINITY, -INFINITY}; }
// Of 8 values, of which those beyond 2^126 become it.
__device__ __forceinline__ Range range_of(float (&x)[8]) {
  Range r = no_values();
  float odd = 0.0f;  // 0 times a value is 0 unless that is infinite or not a number
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    r.lo = fminf(r.lo, x[i]);
    r.hi = fmaxf(r.hi, x[i]);
    odd = fmaf(x[i], 0.0f, odd);
  }
  if (!(odd == 0.0f && r.hi <= kMost && r.lo >= -kMost)) {
    r = no_values();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bool nan = isnan(x[i]);
      x[i] = fminf(fmaxf(x[i], -kMost), kMost);
      r.lo = fminf(r.lo, x[i]);
      r.hi = fmaxf(r.hi, nan ? INFINITY : x[i]);
    }
  }
  return r;
}

struct Scale {
  float s, z, inv;  // inv: 1 / s, 0 for a scale of 0
};
__device__ __forceinline__ Scale scale_of(const Range& r) {
  Scale q;
  const bool nan = r.hi == INFINITY;
  const float lo = nan ? 0.0f : r.lo, hi = nan ? 0.0f : r.hi;
  // (one rounding of the sum, so that a centre next to zero keeps its precision)
  q.z = __bfloat162float(__float2bfloat16_rn(fmaf(lo, 7.0f / 16.0f, hi * 0.5f) * (16.0f / 15.0f)));
  // a seventh, by a quotient corrected by its remainder (as in encode8; a range that is too
  // small for it to be exact becomes 0)
  const float above = hi - q.z, seventh = above * (1.0f / 7.0f);
  q.s = __bfloat162float(__float2bfloat16_ru(fmaxf(fmaf(fmaf(-seventh, 7.0f, above), 1.0f / 7.0f, seventh), (q.z - lo) * 0.125f)));
  if (!(q.s >= kLeastScale)) q.s = 0.0f;
  q.inv = q.s > 0.0f ? 1.0f / q.s : 0.0f;
  if (nan) q.s = __uint_as_float(0x7fc00000u);  // every value of the group reads as NaN
  return q;
}
__device__ __forceinline__ uint16_t bf16_bits(float exact) { return static_cast<uint16_t>(__float_as_uint(exact) >> 16); }

// Codes of 8 neighbouring channels.  The quotient is corrected by its remainder
// (Markstein, IBM J. Res. Dev. 34, 1990), so that it rounds as the division does: bf16
// values lie halfway between two codes often enough (times 1 / s alone, 2 of 1000 codes
// of random bf16 values differed from the definition's).
__device__ __forceinline__ uint32_t encode8(const float (&x)[8], const Scale& q) {
  uint32_t w = 0u - 0x3f400000u;  // what the upper bits of 8 terms of kRound add up to
  const float2 less = make_float2(-q.z, -q.z), inv = make_float2(q.inv, q.inv), by = make_float2(-q.s, -q.s), round = make_float2(kRound, kRound);
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 t = add_pair(make_float2(x[i], x[i + 1]), less), a = mul_pair(t, inv);
    const float2 c = add_pair(fma_pair(fma_pair(a, by, t), inv, a), round);  // from -8 to 7 by the choice of z and s
    w += __float_as_uint(c.x) << (4 * i);
    w += __float_as_uint(c.y) << (4 * i + 4);
  }
  return w;
}
__device__ __forceinline__ void decode8(uint32_t w, float s, float z, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float a = __uint_as_float(((w >> (4 * i)) & 15u) | 0x4b000000u), b = __uint_as_float(((w >> (4 * i + 4)) & 15u) | 0x4b000000u);
    const float2 c = add_pair(make_float2(a, b), make_float2(-8388616.0f, -8388616.0f));  // 2^23 + 8: the codes, exactly
    const float2 v = fma_pair(make_float2(s, s), c, make_float2(z, z));
    x[i] = v.x;
    x[i + 1] = v.y;
  }
}

// Scale and centre of group g of a row.
__device__ __forceinline__ float2 load_scale(const void* scales, int64_t row, int head_dim, int g) {
  const unsigned short* p = reinterpret_cast<const unsigned short*>(scales) + row * record(head_dim);
  return make_float2(bf16_bits_to_float(__ldg(p + g)), bf16_bits_to_float(__ldg(p + head_dim / kQuantGroup + g)));
}
__device__ __forceinline__ void store_scale(void* scales, int64_t row, int head_dim, int g, const Scale& q) {
  uint16_t* p = static_cast<uint16_t*>(scales) + row * record(head_dim);
  p[g] = bf16_bits(q.s);
  p[head_dim / kQuantGroup + g] = bf16_bits(q.z);
}

}  // namespace int4
}  // namespace hs
