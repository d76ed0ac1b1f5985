// Append of any number of new tokens per request to the paged cache: Q and K
// rotated by their positions on the way, K and V written into their pages in
// the cache's format, the min/max summaries of the touched blocks kept current
// ("KV 稀疏化" wiki §5, Quest).  Rotation of a pair (a, b) by its angle:
//   a' = a cos - b sin,  b' = b cos + a sin
// in fp32, rounded once to what is stored.
//
// Block-scaled e4m3 (one scale per page): the scale is the smallest power of
// two s with amax <= 448 s over the page's finite values.  A power of two,
// because a page that is still being filled may have to raise its scale: codes
// written earlier are then multiplied by 2^-n, which loses only what falls
// under the smallest e4m3 step, while any other factor would round every code
// anew.  e4m3 is a floating-point format, so a finer scale would not improve
// its relative precision.  Quantisation with one scale is monotone, so the
// summary of the stored values is the stored image of the rows' min and max.
//
// A thread holds 16 channels of a row as two vectors of 8 chosen so that both
// members of every rotated pair are its own.  One launch either way:
//   any number of rows per request: one warp or four take a unit, one (touched
//     block, kv head, K or V).  They own the page and its scale, so units exchange
//     nothing; rows are held, as read, or read again while the scale is found
//     (rotated twice: held rotated, their registers cost the occupancy that streams
//     Q).  Other CTAs rotate Q: a warp takes 16 heads of a few consecutive rows, and
//     reads a row's cos and sin once for the 16.
//     Memory-bound: prompts of 16 requests of up to 4096 tokens, 32 / 4 heads of 128
//     channels, block-scaled, 859 MB: 131 us, 0.98 of the copy rate; 8 prompts in bf16
//     pages 1.00; with 8 query heads on 8 kv heads 0.78, and 0.54 for both e4m3 kinds
//     (68 us): there the K and V units' instructions count (two rotations, minimum and
//     maximum of every channel: 46 M, 0.58 of the issue slots, the 20 warps of an SM
//     waiting for their loads in between).
//   one row per request: the D / 16 threads of a row take its K and V, so a warp
//     holds several (request, kv head) pairs; the row's thread holds the channels
//     of the summary too, and nothing is exchanged but the row's largest value.
//     Latency-bound: seq_lens, page table, then everything else at once; 256
//     requests x 4 kv heads 3.3 us, block-scaled 3.5.  A page whose scale grows has its
//     earlier rows rewritten by the D / 16 threads alone, K and then V: where the pages
//     of all 256 requests grow at once 10 us with 16-token pages, 30 with 64, 118 with
//     256.
#include <float.h>

#include "hs_internal.h"

namespace hs {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kQHeads = 16;  // heads of one row that a warp rotates

// Largest i in [0, n) with key(i) <= x, for nondecreasing keys with key(0) <= x
// (0 if there is none): 32 probes a round.  All 32 lanes must call it.
template <typename F>
__device__ __forceinline__ int last_not_above(int n, int x, int lane, F key) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + step * (lane + 1);
    const bool below = at < hi && key(at) <= x;
    lo += step * __popc(__ballot_sync(0xffffffffu, below));
    hi = min(hi, lo + step);
  }
  return lo;
}

// Eight f32 or bf16 values as they lie in memory.
template <bool F32>
struct Raw8 {
  uint4 v[F32 ? 2 : 1];
  // (plain loads: Q may be rotated in place, next to K and V in the same rows)
  __device__ __forceinline__ void load(const uint8_t* p) {
    v[0] = reinterpret_cast<const uint4*>(p)[0];
    if constexpr (F32) v[1] = reinterpret_cast<const uint4*>(p)[1];
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t r[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
    if constexpr (F32) {
      const uint32_t q[4] = {v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = __uint_as_float(r[i]);
        x[4 + i] = __uint_as_float(q[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(r[i] << 16);
        x[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
      }
    }
  }
};

// Eight f32 or bf16 values.  INPUT: nothing in the kernel writes them or next to
// them.
template <bool F32, bool INPUT = true>
__device__ __forceinline__ void load8(const void* p, int64_t at, float (&x)[8]) {
  if constexpr (F32) {
    const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
    const float4 u = INPUT ? __ldg(s) : s[0], w = INPUT ? __ldg(s + 1) : s[1];
    x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
    x[4] = w.x; x[5] = w.y; x[6] = w.z; x[7] = w.w;
  } else {
    const uint4* s = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
    const uint4 u = INPUT ? __ldg(s) : *s;
    const uint32_t r[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(r[i] << 16);
      x[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
    }
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

template <bool F32>
__device__ __forceinline__ void store8(void* p, int64_t at, const float (&x)[8]) {
  if constexpr (F32) {
    float4* d = reinterpret_cast<float4*>(static_cast<float*>(p) + at);
    d[0] = make_float4(x[0], x[1], x[2], x[3]);
    d[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at) =
        make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
  }
}

__device__ __forceinline__ uint2 encode8(const float (&x)[8], float inv) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * i] * inv, x[2 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

__device__ __forceinline__ float decode1(uint32_t code) { return e4m3x2_to_float2(static_cast<uint16_t>(code)).x; }

// The value that the code of x (at scale s) stands for.
__device__ __forceinline__ float as_stored(float x, float inv, float s) {
  const __nv_fp8x2_storage_t c = __nv_cvt_float2_to_fp8x2(make_float2(x * inv, 0.0f), __NV_SATFINITE, __NV_E4M3);
  return decode1(c) * s;
}

constexpr float kMinScale = 6.018531076210112e-36f;  // 2^-117: code times scale stays a normal number

// Smallest power of two s >= 2^-117 with amax <= 448 s (amax finite).
__device__ __forceinline__ float block_scale(float amax) {
  if (!(amax > 448.0f * kMinScale)) return kMinScale;
  // amax = 2^e m with m in [1, 2); 448 = 2^8 * 1.75
  const uint32_t u = __float_as_uint(amax);
  const int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// The two 8-channel vectors of slot s of a row, and their rotation.
struct Slot {
  int ca, cb;    // first channels
  bool rotated;  // by angles 8 s .. 8 s + 7
};
__device__ __forceinline__ Slot slot_of(int s, int rotary, bool interleaved) {
  Slot t;
  t.rotated = 16 * s < rotary;
  const bool split = t.rotated && !interleaved;
  t.ca = split ? 8 * s : 16 * s;
  t.cb = split ? 8 * s + rotary / 2 : 16 * s + 8;
  return t;
}

struct Angles {
  float c[8], s[8];
};
__device__ __forceinline__ void load_angles(const float* cos_sin, int rotary, int64_t pos, int s, Angles& t) {
  const float* row = cos_sin + pos * rotary + 8 * s;
  load8<true>(row, 0, t.c);
  load8<true>(row, rotary / 2, t.s);
}
template <bool INTERLEAVED>  // (at run time both forms would be computed and one kept)
__device__ __forceinline__ void rotate(float (&a)[8], float (&b)[8], const Angles& t) {
  if constexpr (INTERLEAVED) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = a[2 * i], y = a[2 * i + 1], z = b[2 * i], w = b[2 * i + 1];
      a[2 * i] = fmaf(x, t.c[i], -(y * t.s[i]));
      a[2 * i + 1] = fmaf(y, t.c[i], x * t.s[i]);
      b[2 * i] = fmaf(z, t.c[4 + i], -(w * t.s[4 + i]));
      b[2 * i + 1] = fmaf(w, t.c[4 + i], z * t.s[4 + i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = a[i], y = b[i];
      a[i] = fmaf(x, t.c[i], -(y * t.s[i]));
      b[i] = fmaf(y, t.c[i], x * t.s[i]);
    }
  }
}

// Units for the touched blocks: with offsets, request b's blocks have the slots
// from offsets[b] / B + 2 b on.
int64_t kv_units_of(const KvView& kv, const AppendTokensArgs& a) {
  return (a.rows / kv.block + 2 * static_cast<int64_t>(kv.batch)) * kv.hkv * 2;
}
// Rows a warp rotates 16 heads of: more than one only where there are warps
// enough without that (8000 tokens of 32 heads: 4 rows 38.0 us, one 39.3; 2000 tokens
// 13.1 and 11.9).
int q_rows_of(const KvView& kv, const AppendTokensArgs& a) {
  return a.offsets && a.rows * ceil_div(kv.hq, kQHeads) >= 8000 ? 4 : 1;
}
int64_t q_units_of(const KvView& kv, const AppendTokensArgs& a) {
  const int n = q_rows_of(kv, a);
  return a.q ? (a.rows + n - 1) / n * ceil_div(kv.hq, kQHeads) : 0;
}

// Request of new row `row` and its position in the cache; false: no such row.
__device__ __forceinline__ bool place_of_row(const KvView& kv, const AppendTokensArgs& a, int64_t row, int b, int64_t* p) {
  int64_t behind = 1;  // tokens from this row's to the end of its request
  if (a.offsets) {
    const int64_t o0 = __ldg(a.offsets + b), o1 = __ldg(a.offsets + b + 1);
    // behind the last request, or offsets that are reported by the K and V units
    if (row < o0 || row >= o1 || o1 > a.rows || o1 - o0 > __ldg(kv.seq_lens + b)) return false;
    behind = o1 - row;
  }
  *p = static_cast<int64_t>(__ldg(kv.seq_lens + b)) - behind;
  return *p >= 0;
}

// kQHeads heads of rows [row, row_end).
template <int D, bool F32, bool INTERLEAVED>
__device__ void rotate_q(const KvView& kv, const AppendTokensArgs& a, int h0, int64_t row, int64_t row_end, int lane,
                         unsigned* err) {
  constexpr int TPR = D / 16, HPP = 32 / TPR, N = kQHeads / HPP;  // threads per head, heads per step, steps
  constexpr int E = F32 ? 4 : 2;
  const int s = lane % TPR, h = h0 + lane / TPR;
  const Slot t = slot_of(s, a.rotary, INTERLEAVED);
  const uint8_t* q = static_cast<const uint8_t*>(a.q) + (row * a.q_stride + h * D) * E;
  uint8_t* out = static_cast<uint8_t*>(a.q_out) + (row * a.q_out_stride + h * D) * E;
  Raw8<F32> x[N], y[N];
  const auto read = [&]() {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (h + i * HPP < kv.hq) {
        x[i].load(q + (i * HPP * D + t.ca) * E);
        y[i].load(q + (i * HPP * D + t.cb) * E);
      }
  };
  read();  // ahead of everything that takes lookups
  int b = static_cast<int>(row);
  if (a.offsets) b = last_not_above(kv.batch, static_cast<int>(row), lane, [&](int i) { return __ldg(a.offsets + i); });
  for (;;) {
    int64_t p, pos = 0;
    bool ok = place_of_row(kv, a, row, b, &p);
    if (ok) {
      pos = a.positions ? __ldg(a.positions + row) : p;
      if (a.rotary > 0 && (pos < 0 || pos >= a.table_rows)) {
        if (lane == 0) set_error(err, HS_EBIT_POSITION);
        ok = false;
      }
    }
    if (ok) {
      Angles ang;
      if (t.rotated) load_angles(a.cos_sin, a.rotary, pos, s, ang);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float u[8], w[8];
        x[i].get(u);
        y[i].get(w);
        if (t.rotated) rotate<INTERLEAVED>(u, w, ang);
        if (h + i * HPP < kv.hq) {
          store8<F32>(out + (i * HPP * D + t.ca) * E, 0, u);
          store8<F32>(out + (i * HPP * D + t.cb) * E, 0, w);
        }
      }
    }
    if (++row >= row_end) return;
    q += a.q_stride * E;
    out += a.q_out_stride * E;
    read();
    if (a.offsets)
      while (b + 1 < kv.batch && row >= __ldg(a.offsets + b + 1)) ++b;
    else
      b = static_cast<int>(row);
  }
}

// What 8 codes stand for at scale s.
__device__ __forceinline__ void decode8(uint2 c, float s, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = e4m3x2_to_float2(static_cast<uint16_t>((i < 2 ? c.x : c.y) >> (16 * (i & 1))));
    x[2 * i] = f.x * s;
    x[2 * i + 1] = f.y * s;
  }
}

// x / s for each x, rounded as IEEE division rounds it.  Where s is of ordinary size
// after Markstein (IBM J. Res. Dev. 34, 1990): with r = 1 / s rounded, the remainder
// of x r corrects it to the rounded quotient.  (Compared with division on the host
// for every significand of s and the three x next to each border of a code's
// neighbours, where a code could differ: 8 10^8 quotients, all the same.)  The
// remainder is exact for |x| >= 2^-101; a smaller x has a quotient under 2^-40, which
// no code shows but by its sign.  The remainder is taken as q s - x and subtracted, so
// that a quotient of -0 stays one (0 - 0 is +0, and -0 - (+0) is -0).  Prompts of 8 / 8 heads 95 us, with divisions 114 (before P = 2).
__device__ __forceinline__ void divide8(float (&x)[8], float s) {
  if (s >= 8.673617379884035e-19f && s <= 1.152921504606847e18f) {  // 2^-60, 2^60
    const float r = 1.0f / s;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const float q = x[c] * r;
      x[c] = fmaf(-fmaf(q, s, -x[c]), r, q);
    }
  } else {
#pragma unroll
    for (int c = 0; c < 8; ++c) x[c] = x[c] / s;
  }
}

// The grouped format: every 32-channel group its own scale (amax / 448).  A row's
// TPR neighbouring threads call it together; `part` is their D / 32 words of
// shared memory.  Stores the codes and scales and leaves in u, w what they stand
// for.
template <int D, bool INTERLEAVED>
__device__ __forceinline__ void store_grouped(void* pages, float* scales, int64_t row, int s, const Slot& t, int rotary, bool live,
                                              unsigned* part, float (&u)[8], float (&w)[8]) {
  float ga = 0.0f, gb = 0.0f;  // the largest magnitudes of the vectors' groups
  if (live) {
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      ga = fmaxf(ga, fabsf(u[c]));
      gb = fmaxf(gb, fabsf(w[c]));
    }
  }
  const bool split = !INTERLEAVED && t.rotated;
  const bool neighbours = INTERLEAVED || rotary % 64 == 0;
  if (neighbours) {  // a group is two threads' vectors, or (split) one vector of four threads
    if (!split) ga = gb = fmaxf(ga, gb);
    ga = fmaxf(ga, __shfl_xor_sync(0xffffffffu, ga, 1));
    gb = fmaxf(gb, __shfl_xor_sync(0xffffffffu, gb, 1));
    if constexpr (!INTERLEAVED) {
      const float a2 = __shfl_xor_sync(0xffffffffu, ga, 2), b2 = __shfl_xor_sync(0xffffffffu, gb, 2);
      if (split) {
        ga = fmaxf(ga, a2);
        gb = fmaxf(gb, b2);
      }
    }
  } else {
    if (s < D / kQuantGroup) part[s] = 0u;
    __syncwarp();
    if (live) {
      atomicMax(&part[t.ca / kQuantGroup], __float_as_uint(ga));  // a maximum: the order does not matter
      atomicMax(&part[t.cb / kQuantGroup], __float_as_uint(gb));
    }
    __syncwarp();
    ga = __uint_as_float(part[t.ca / kQuantGroup]);
    gb = __uint_as_float(part[t.cb / kQuantGroup]);
    __syncwarp();
  }
  if (!live) return;
  const float sa = ga > 0.0f ? ga / 448.0f : 1.0f, sb = gb > 0.0f ? gb / 448.0f : 1.0f;
  divide8(u, sa);  // as the quantiser of whole rows does
  divide8(w, sb);
  uint8_t* dst = static_cast<uint8_t*>(pages) + row * D;
  const uint2 cu = encode8(u, 1.0f), cw = encode8(w, 1.0f);
  *reinterpret_cast<uint2*>(dst + t.ca) = cu;
  *reinterpret_cast<uint2*>(dst + t.cb) = cw;
  // the thread with a group's first channel has its scale
  if (t.ca % kQuantGroup == 0) scales[row * (D / kQuantGroup) + t.ca / kQuantGroup] = sa;
  if (t.cb % kQuantGroup == 0) scales[row * (D / kQuantGroup) + t.cb / kQuantGroup] = sb;
  decode8(cu, sa, u);
  decode8(cw, sb, w);
}

// Stores a row of an f32 or bf16 cache and leaves in u, w what it holds.
template <int D, int KIND>
__device__ __forceinline__ void store_plain(void* pages, int64_t row, const Slot& t, float (&u)[8], float (&w)[8]) {
  store8<KIND == HS_KV_F32>(pages, row * D + t.ca, u);
  store8<KIND == HS_KV_F32>(pages, row * D + t.cb, w);
  if constexpr (KIND == HS_KV_BF16) {
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      u[c] = __bfloat162float(__float2bfloat16_rn(u[c]));
      w[c] = __bfloat162float(__float2bfloat16_rn(w[c]));
    }
  }
}

// Largest magnitude among the values and m (NaN aside), and the same without
// infinities.
__device__ __forceinline__ float widen_any(float m, const float (&u)[8], const float (&w)[8]) {
#pragma unroll
  for (int c = 0; c < 8; ++c) m = fmaxf(m, fmaxf(fabsf(u[c]), fabsf(w[c])));
  return m;
}
__device__ __forceinline__ float widen_finite(float m, const float (&u)[8], const float (&w)[8]) {
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const float p = fabsf(u[c]), q = fabsf(w[c]);
    m = fmaxf(m, p <= FLT_MAX ? p : 0.0f);
    m = fmaxf(m, q <= FLT_MAX ? q : 0.0f);
  }
  return m;
}

// 16 codes times f (a page whose scale grows)
__device__ __forceinline__ uint4 rescaled(uint4 v, float f) {
  const uint32_t in[4] = {v.x, v.y, v.z, v.w};
  uint32_t out[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const float2 lo = e4m3x2_to_float2(static_cast<uint16_t>(in[c])), hi = e4m3x2_to_float2(static_cast<uint16_t>(in[c] >> 16));
    out[c] = __nv_cvt_float2_to_fp8x2(make_float2(lo.x * f, lo.y * f), __NV_SATFINITE, __NV_E4M3) |
             static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(hi.x * f, hi.y * f), __NV_SATFINITE, __NV_E4M3)) << 16;
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

// ---- any number of rows per request ----
// A unit is one touched block of one kv head, K or V.  One warp takes it, or the
// CTA's four: the page's rows are read in passes of 32 / (D / 16) rows a warp, P
// passes at a time, and one warp takes pages of up to 4 passes.  (8 requests of up to
// 4096 tokens, 8 kv heads, block-scaled: 4 passes, 16-token pages, by one warp 105 us,
// by four 132; 8 passes, 32-token pages, by four warps 77, by two 99; and four warps
// taking 128-token pages in turns 67, eight at once 76.)
//
// Block-scaled, the rows of one turn are held, as read, until the scale is known, and
// those of more turns are read once more, from the caches.  P = 2 leaves registers for
// 640 threads on an SM instead of 512: prompts of 16 requests 131 us, P = 4, all rows
// of a page held, 134; 8 / 8 heads 70 and 79.  Where all units run at once that counts
// for nothing and holding saves the second reading: a chunk of 2000 tokens 12.2 us,
// P = 2 13.2.  Grouped e4m3: P = 2, 8 / 8 heads 71 us, P = 4 95.  bf16 and f32 take P = 4:
// bf16 at 640 threads, whose 96 registers spill 112 bytes (188 where one warp takes a
// page), 56 us, at 512 without spills 60; f32 at 512 (up to 36 bytes) 89, at 384 97.
constexpr int threads_per_sm(int kind, int p) {
  return kind == HS_KV_F32 || (kind == HS_KV_FP8E4M3_BLOCK && p == 4) ? 512 : 640;
}

template <int D, int KIND, bool INTERLEAVED, int UW, int P>
__global__ __launch_bounds__(kThreads, threads_per_sm(KIND, P) / kThreads) void append_rows_kernel(
    KvView kv, AppendTokensArgs a, int kv_units, uint64_t mix, int q_units, int q_rows, unsigned* err) {
  constexpr bool F32 = KIND == HS_KV_F32;
  static_assert(UW == 1 || UW == kWarps);
  constexpr int kUnits = kWarps / UW;  // of a CTA
  constexpr int TPR = D / 16, RPP = UW * 32 / TPR;  // threads per row, rows per pass of a unit
  __shared__ float s_mn[kWarps][D], s_mx[kWarps][D];
  __shared__ float s_amax[kWarps];
  __shared__ int s_any[kWarps];
  __shared__ unsigned s_group[kWarps * 32 / TPR][D / kQuantGroup];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // ---- K and V units are spread over the first `span` CTAs, the others rotate Q ----
  // (mix: K and V CTAs per CTA, in 2^-32; divisions are in 32 bits: they are most
  // of a unit's fixed work)
  const int kv_ctas = (kv_units + kUnits - 1) / kUnits;
  const int cta = static_cast<int>(min((blockIdx.x * mix) >> 32, static_cast<uint64_t>(kv_ctas)));
  if (static_cast<int>(min(((blockIdx.x + uint64_t(1)) * mix) >> 32, static_cast<uint64_t>(kv_ctas))) == cta) {
    const int q = static_cast<int>(blockIdx.x - cta) * kWarps + warp;
    if (q >= q_units) return;
    const int chunks = ceil_div(kv.hq, kQHeads), r = q / chunks;
    rotate_q<D, F32, INTERLEAVED>(kv, a, (q - r * chunks) * kQHeads, static_cast<int64_t>(r) * q_rows,
                                  min(a.rows, (r + int64_t(1)) * q_rows), lane, err);
    return;
  }
  // ---- which block ----
  const int first_warp = warp / UW * UW, tid = threadIdx.x - first_warp * 32;  // the unit's first warp, the thread in it
  const auto unit_sync = [&]() {
    if constexpr (UW == 1)
      __syncwarp();
    else
      __syncthreads();
  };
  const int unit = cta * kUnits + first_warp / UW;
  if (unit >= kv_units) return;
  const bool is_k = (unit & 1) == 0;
  const int slot = (unit >> 1) / kv.hkv, kvh = (unit >> 1) - slot * kv.hkv;
  const int B = kv.block;
  const auto bad = [&](int o0, int o1, int L) { return o0 < 0 || o1 < o0 || o1 > a.rows || o1 - o0 > max(L, 0); };
  // The search below finds every request with rows only where the offsets ascend, so
  // each request is checked apart from it, by as many of the last units (there are four
  // or more for each request, and the last ones have spare slots).
  const int checked = kv_units - 1 - unit;
  if (tid == 0 && checked < kv.batch &&
      bad(__ldg(a.offsets + checked), __ldg(a.offsets + checked + 1), __ldg(kv.seq_lens + checked)))
    set_error(err, HS_EBIT_BLOCK_RANGE);
  // request b has the slots from offsets[b] / B + 2 b on: enough for every block
  // its rows can touch, wherever in a block they begin
  const int shift = (B & (B - 1)) == 0 ? 31 - __clz(B) : -1;
  const auto blocks = [&](int rows) { return shift >= 0 ? rows >> shift : rows / B; };
  const int b = last_not_above(kv.batch, slot, lane, [&](int i) { return blocks(__ldg(a.offsets + i)) + 2 * i; });
  const int o0 = __ldg(a.offsets + b), o1 = __ldg(a.offsets + b + 1);
  const int L = __ldg(kv.seq_lens + b);
  if (bad(o0, o1, L)) return;
  const int n = o1 - o0, x = slot - (blocks(o0) + 2 * b);
  if (x < 0 || n == 0) return;
  const int first = L - n;  // cache position of the request's first new row
  const int j = blocks(first) + x;
  if (j > blocks(L - 1)) return;
  const int64_t pair = static_cast<int64_t>(b) * kv.hkv + kvh;
  if (j >= kv.max_blocks) {
    if (tid == 0) set_error(err, HS_EBIT_BLOCK_RANGE);
    return;
  }
  const int ra = max(0, first - j * B), rb = min(B, L - j * B);  // rows of the page that are new
  const void* src = is_k ? a.k : a.v;
  const int64_t stride = is_k ? a.k_stride : a.v_stride;
  const int64_t src0 = o0 + (j * B - first);  // + page row = source row
  void* pages = const_cast<void*>(is_k ? kv.k_pages : kv.v_pages);
  float* scales = const_cast<float*>(is_k ? kv.k_scales : kv.v_scales);
  const int rotary = is_k ? a.rotary : 0;
  const bool box = is_k && a.smin != nullptr;
  const int s = tid % TPR, rs = tid / TPR;
  const Slot t = slot_of(s, a.rotary, INTERLEAVED);

  // Page rows r0 + i RPP + rs, as they lie in memory: every load before the first
  // use; rows past the end repeat the last.
  constexpr int E = F32 ? 4 : 2;
  Raw8<F32> xa[P], xb[P];
  const uint8_t* from = static_cast<const uint8_t*>(src) + (src0 * stride + kvh * D) * E;
  const auto read = [&](int r0) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const uint8_t* p = from + min(r0 + i * RPP + rs, rb - 1) * stride * E;
      xa[i].load(p + t.ca * E);
      xb[i].load(p + t.cb * E);
    }
  };
  read(ra);  // (ahead of the page's lookup)
  const int page = kv.page_table[pair * kv.max_blocks + j];
  if (page < 0 || page >= kv.num_pages) {
    if (tid == 0) set_error(err, HS_EBIT_PAGE_RANGE);
    return;
  }
  const int64_t row0 = static_cast<int64_t>(page) * B;
  // Row r (of those that were read, the i-th), rotated; false: no such row, or
  // its position has no angles.
  const auto turned = [&](int r, const Raw8<F32>& va, const Raw8<F32>& vb, float (&u)[8], float (&w)[8]) {
    if (r >= rb) return false;
    va.get(u);
    vb.get(w);
    if (rotary > 0) {
      const int64_t pos = a.positions ? __ldg(a.positions + src0 + r) : static_cast<int64_t>(j) * B + r;
      if (pos < 0 || pos >= a.table_rows) {
        set_error(err, HS_EBIT_POSITION);
        return false;
      }
      if (t.rotated) {
        Angles ang;
        load_angles(a.cos_sin, rotary, pos, s, ang);
        rotate<INTERLEAVED>(u, w, ang);
      }
    }
    return true;
  };

  float mn[16], mx[16];
#pragma unroll
  for (int c = 0; c < 16; ++c) {
    mn[c] = INFINITY;
    mx[c] = -INFINITY;
  }
  bool any = false;
  float amax = 0.0f;
  for (int r0 = ra; r0 < rb; r0 += P * RPP) {
    if (r0 > ra) read(r0);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      float u[8], w[8];
      const int r = r0 + i * RPP + rs;
      const bool on = turned(r, xa[i], xb[i], u, w);
      any |= on;
      if constexpr (KIND == HS_KV_FP8E4M3_G32) {
        store_grouped<D, INTERLEAVED>(pages, scales, row0 + r, s, t, a.rotary, on, s_group[threadIdx.x / TPR], u, w);
      } else if constexpr (KIND == HS_KV_FP8E4M3_BLOCK) {
        if (on && !box) amax = widen_any(amax, u, w);
      } else {
        if (on) store_plain<D, KIND>(pages, row0 + r, t, u, w);
      }
      if (box && on) {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          mn[c] = fminf(mn[c], u[c]);
          mx[c] = fmaxf(mx[c], u[c]);
          mn[8 + c] = fminf(mn[8 + c], w[c]);
          mx[8 + c] = fmaxf(mx[8 + c], w[c]);
        }
      }
    }
  }

  float scale = 1.0f, inv = 1.0f;
  bool grown = false;
  if constexpr (KIND == HS_KV_FP8E4M3_BLOCK) {
    const float held = ra > 0 ? scales[page] : 0.0f;  // read by every thread before one of them writes it (below)
    if (box && any) {  // the box has the largest magnitude in it
#pragma unroll
      for (int c = 0; c < 16; ++c) amax = fmaxf(amax, mn[c] <= mx[c] ? fmaxf(-mn[c], mx[c]) : 0.0f);
    }
    const auto over_unit = [&](float m) {
      m = warp_max(m);
      if constexpr (UW > 1) {
        if (lane == 0) s_amax[warp] = m;
        unit_sync();
#pragma unroll
        for (int i = 0; i < UW; ++i) m = fmaxf(m, s_amax[first_warp + i]);
      }
      return m;
    };
    amax = over_unit(amax);
    const bool again = rb - ra > P * RPP;  // more rows than are held: read once more, from the caches
    if (amax == INFINITY) {  // the scale goes by the finite values
      amax = 0.0f;
      for (int r0 = ra; r0 < rb; r0 += P * RPP) {
        if (again) read(r0);
#pragma unroll
        for (int i = 0; i < P; ++i) {
          float u[8], w[8];
          if (turned(r0 + i * RPP + rs, xa[i], xb[i], u, w)) amax = widen_finite(amax, u, w);
        }
      }
      unit_sync();
      amax = over_unit(amax);
    }
    scale = block_scale(amax);
    if (ra > 0) {
      grown = !(held >= scale);  // (a scale that is not a number is replaced)
      if (!grown) scale = held;
    }
    inv = 1.0f / scale;
    if (grown) {  // the rows already there, at the new scale
      const float f = held > 0.0f ? held * inv : 0.0f;
      for (int r = rs; r < ra; r += RPP) {
        uint4* p = reinterpret_cast<uint4*>(static_cast<uint8_t*>(pages) + (row0 + r) * D + 16 * s);
        *p = rescaled(*p, f);
      }
    }
    if constexpr (UW == 1) __syncwarp();
    if (tid == 0 && (ra == 0 || grown)) scales[page] = scale;
    for (int r0 = ra; r0 < rb; r0 += P * RPP) {
      if (again) read(r0);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        float u[8], w[8];
        const int r = r0 + i * RPP + rs;
        if (turned(r, xa[i], xb[i], u, w)) {
          uint8_t* dst = static_cast<uint8_t*>(pages) + (row0 + r) * D;
          *reinterpret_cast<uint2*>(dst + t.ca) = encode8(u, inv);
          *reinterpret_cast<uint2*>(dst + t.cb) = encode8(w, inv);
        }
      }
    }
  }
  if (!box) return;

  // ---- the block's summary ----
#pragma unroll
  for (int off = TPR; off < 32; off <<= 1)
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      mn[c] = fminf(mn[c], __shfl_xor_sync(0xffffffffu, mn[c], off));
      mx[c] = fmaxf(mx[c], __shfl_xor_sync(0xffffffffu, mx[c], off));
    }
  if (lane < TPR) {
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      const int d = (c < 8 ? t.ca : t.cb) + (c & 7);
      s_mn[warp][d] = mn[c];
      s_mx[warp][d] = mx[c];
    }
  }
  any = __any_sync(0xffffffffu, any);
  if (lane == 0) s_any[warp] = any ? 1 : 0;
  unit_sync();  // (also: the page's rows are written)
  int rows_written = 0;
#pragma unroll
  for (int i = 0; i < UW; ++i) rows_written |= s_any[first_warp + i];
  if (!rows_written) return;  // every row's position was out of range
#pragma unroll
  for (int d = tid; d < D; d += UW * 32) {
    float lo = s_mn[first_warp][d], hi = s_mx[first_warp][d];
#pragma unroll
    for (int i = 1; i < UW; ++i) {
      lo = fminf(lo, s_mn[first_warp + i][d]);
      hi = fmaxf(hi, s_mx[first_warp + i][d]);
    }
    if constexpr (KIND == HS_KV_FP8E4M3_BLOCK) {
      if (lo <= hi) {  // (else only NaN)
        lo = as_stored(lo, inv, scale);
        hi = as_stored(hi, inv, scale);
      }
      if (grown)  // the earlier rows' codes may have been rounded: their box is taken anew
        for (int r = 0; r < ra; ++r) {
          const float v = decode1(static_cast<const uint8_t*>(pages)[(row0 + r) * D + d]) * scale;
          lo = fminf(lo, v);
          hi = fmaxf(hi, v);
        }
    }
    const int64_t o = (pair * kv.max_blocks + j) * D + d;
    const bool keep = ra > 0 && !grown;
    if constexpr (F32) {
      float* pn = static_cast<float*>(a.smin) + o;
      float* px = static_cast<float*>(a.smax) + o;
      *pn = keep ? fminf(*pn, lo) : lo;
      *px = keep ? fmaxf(*px, hi) : hi;
    } else {
      __nv_bfloat16* pn = static_cast<__nv_bfloat16*>(a.smin) + o;
      __nv_bfloat16* px = static_cast<__nv_bfloat16*>(a.smax) + o;
      lo = __bfloat162float(__float2bfloat16_rd(lo));  // outward; exact for values that are bf16 already
      hi = __bfloat162float(__float2bfloat16_ru(hi));
      *pn = __float2bfloat16_rn(keep ? fminf(__bfloat162float(*pn), lo) : lo);
      *px = __float2bfloat16_rn(keep ? fmaxf(__bfloat162float(*px), hi) : hi);
    }
  }
}

// ---- one row per request ----
// Eight channels of a summary row, widened to lo / hi (or started afresh).
template <bool F32>
__device__ __forceinline__ void widen_box(void* smin, void* smax, int64_t at, bool keep, float (&lo)[8], float (&hi)[8]) {
  if (keep) {
    float p[8], q[8];
    load8<F32, false>(smin, at, p);
    load8<F32, false>(smax, at, q);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      lo[c] = fminf(p[c], lo[c]);
      hi[c] = fmaxf(q[c], hi[c]);
    }
  }
  store8<F32>(smin, at, lo);
  store8<F32>(smax, at, hi);
}

template <int D, int KIND, bool INTERLEAVED>
__global__ __launch_bounds__(kThreads) void append_one_kernel(KvView kv, AppendTokensArgs a, int kv_ctas, unsigned* err) {
  constexpr bool F32 = KIND == HS_KV_F32;
  constexpr int TPR = D / 16, RPC = kThreads / TPR;  // threads per row, rows per CTA
  __shared__ unsigned s_group[RPC][D / kQuantGroup];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (static_cast<int>(blockIdx.x) >= kv_ctas) {
    const int64_t q = static_cast<int64_t>(blockIdx.x - kv_ctas) * kWarps + warp;
    const int chunks = ceil_div(kv.hq, kQHeads);
    const int64_t row = q / chunks;
    if (row < a.rows) rotate_q<D, F32, INTERLEAVED>(kv, a, static_cast<int>(q - row * chunks) * kQHeads, row, row + 1, lane, err);
    return;
  }
  const int s = tid % TPR, rs = tid / TPR;
  const int pairs = kv.batch * kv.hkv;
  const int pair = static_cast<int>(blockIdx.x) * RPC + rs;
  const int b = min(pair, pairs - 1) / kv.hkv, kvh = min(pair, pairs - 1) - b * kv.hkv;
  const Slot t = slot_of(s, a.rotary, INTERLEAVED);
  // the row itself needs no lookup
  float ku[8], kw[8], vu[8], vw[8];
  load8<F32, false>(a.k, b * a.k_stride + kvh * D + t.ca, ku);
  load8<F32, false>(a.k, b * a.k_stride + kvh * D + t.cb, kw);
  load8<F32, false>(a.v, b * a.v_stride + kvh * D + t.ca, vu);
  load8<F32, false>(a.v, b * a.v_stride + kvh * D + t.cb, vw);
  const int B = kv.block, L = __ldg(kv.seq_lens + b);
  const int p = L - 1, j = p / B, r = p - j * B;
  bool live = pair < pairs && L > 0, live_k = false;
  int page = 0;
  if (live) {
    if (j >= kv.max_blocks) {
      set_error(err, HS_EBIT_BLOCK_RANGE);
      live = false;
    } else {
      page = __ldg(kv.page_table + static_cast<int64_t>(pair) * kv.max_blocks + j);
      if (page < 0 || page >= kv.num_pages) {
        set_error(err, HS_EBIT_PAGE_RANGE);
        live = false;
      }
    }
  }
  if (live) {
    live_k = true;
    if (a.rotary > 0) {
      const int64_t pos = a.positions ? __ldg(a.positions + b) : p;
      if (pos < 0 || pos >= a.table_rows) {
        set_error(err, HS_EBIT_POSITION);
        live_k = false;
      } else if (t.rotated) {
        Angles ang;
        load_angles(a.cos_sin, a.rotary, pos, s, ang);
        rotate<INTERLEAVED>(ku, kw, ang);
      }
    }
  }
  const int64_t row0 = static_cast<int64_t>(page) * B, row = row0 + r;
  void* kp = const_cast<void*>(kv.k_pages);
  void* vp = const_cast<void*>(kv.v_pages);
  float* ks = const_cast<float*>(kv.k_scales);
  float* vs = const_cast<float*>(kv.v_scales);
  const bool box = a.smin != nullptr;

  if constexpr (KIND == HS_KV_FP8E4M3_G32) {
    store_grouped<D, INTERLEAVED>(kp, ks, row, s, t, a.rotary, live_k, s_group[rs], ku, kw);
    store_grouped<D, INTERLEAVED>(vp, vs, row, s, t, a.rotary, live, s_group[rs], vu, vw);
  } else if constexpr (KIND == HS_KV_FP8E4M3_BLOCK) {
    float lo[16], hi[16];  // box of the earlier rows, channels 16 s and up, where their codes change
    // The page's scale, the codes and the earlier rows' codes where the scale
    // grows (false); afterwards u, w are what is held.
    const auto store_block = [&](void* pages, float* scales, bool on, bool boxes, float (&u)[8], float (&w)[8]) {
      float amax = on ? widen_finite(0.0f, u, w) : 0.0f;
#pragma unroll
      for (int o = TPR / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      bool kept = true;
      if (on) {
        const float held = r > 0 ? scales[page] : 0.0f;
        float scale = block_scale(amax);
        const bool grown = r > 0 && !(held >= scale);  // (a scale that is not a number is replaced)
        if (r > 0 && !grown) scale = held;
        const float inv = 1.0f / scale;
        if (grown) {
          const float f = held > 0.0f ? held * inv : 0.0f;
          kept = false;
#pragma unroll 4
          for (int i = 0; i < r; ++i) {
            uint4* at = reinterpret_cast<uint4*>(static_cast<uint8_t*>(pages) + (row0 + i) * D + 16 * s);
            const uint4 c = rescaled(*at, f);
            *at = c;
            if (boxes) {
              float x[8], y[8];
              decode8(make_uint2(c.x, c.y), scale, x);
              decode8(make_uint2(c.z, c.w), scale, y);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                lo[e] = fminf(lo[e], x[e]);
                hi[e] = fmaxf(hi[e], x[e]);
                lo[8 + e] = fminf(lo[8 + e], y[e]);
                hi[8 + e] = fmaxf(hi[8 + e], y[e]);
              }
            }
          }
        }
        uint8_t* dst = static_cast<uint8_t*>(pages) + row * D;
        const uint2 cu = encode8(u, inv), cw = encode8(w, inv);
        *reinterpret_cast<uint2*>(dst + t.ca) = cu;
        *reinterpret_cast<uint2*>(dst + t.cb) = cw;
        decode8(cu, scale, u);
        decode8(cw, scale, w);
        __syncwarp(((1u << TPR) - 1u) << (lane / TPR * TPR));  // every thread of the row has read the old scale
        if (s == 0 && (r == 0 || grown)) scales[page] = scale;
      }
      return kept;
    };
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      lo[c] = INFINITY;
      hi[c] = -INFINITY;
    }
    const bool kept = store_block(kp, ks, live_k, box, ku, kw);
    store_block(vp, vs, live, false, vu, vw);
    if (live_k && box && !kept) {
      // the earlier rows' box lies by 16 neighbouring channels to a thread: it
      // goes down first, and the row widens it like any other
      const int64_t at = (static_cast<int64_t>(pair) * kv.max_blocks + j) * D + 16 * s;
      float x[8], y[8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          x[c] = __bfloat162float(__float2bfloat16_rd(lo[8 * h + c]));
          y[c] = __bfloat162float(__float2bfloat16_ru(hi[8 * h + c]));
        }
        widen_box<false>(a.smin, a.smax, at + 8 * h, false, x, y);
      }
    }
    __syncwarp();
  } else {
    if (live_k) store_plain<D, KIND>(kp, row, t, ku, kw);
    if (live) store_plain<D, KIND>(vp, row, t, vu, vw);
  }
  if (!box || !live_k) return;
  const int64_t at = (static_cast<int64_t>(pair) * kv.max_blocks + j) * D;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float x[8], y[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const float v = h ? kw[c] : ku[c];
      // NaN: nothing to widen.  bf16: outward, exact for values that are bf16 already
      x[c] = isnan(v) ? INFINITY : F32 ? v : __bfloat162float(__float2bfloat16_rd(v));
      y[c] = isnan(v) ? -INFINITY : F32 ? v : __bfloat162float(__float2bfloat16_ru(v));
    }
    widen_box<F32>(a.smin, a.smax, at + (h ? t.cb : t.ca), r > 0, x, y);
  }
}

template <int D, int KIND, bool INTERLEAVED, int UW, int P>
cudaError_t launch_rows(const KvView& kv, const AppendTokensArgs& a, int sms, unsigned* err, cudaStream_t st) {
  constexpr int kUnits = kWarps / UW;
  const int64_t kv_units = kv_units_of(kv, a), kv_ctas = (kv_units + kUnits - 1) / kUnits;
  const int64_t q_units = q_units_of(kv, a), ctas = kv_ctas + (q_units + kWarps - 1) / kWarps;
  // K and V units go first where two rounds of them at most fill the GPU: they take
  // longest (a chunk of 2000 tokens 11.9 us, mixed evenly 14.4; 3000 tokens 15.8 and
  // 19.2).  More than that are mixed evenly with the Q units, which keep the memory
  // busy while they look up and reduce (12000 tokens 53.8, K and V first 58.0).
  const int64_t span = kv_ctas <= 2 * static_cast<int64_t>(sms) * (threads_per_sm(KIND, P) / kThreads) ? kv_ctas : ctas;
  const uint64_t mix = ((static_cast<uint64_t>(kv_ctas) << 32) + span - 1) / span;
  return launch_pdl(append_rows_kernel<D, KIND, INTERLEAVED, UW, P>, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), 0, st, kv, a,
                    static_cast<int>(kv_units), mix, static_cast<int>(q_units), q_rows_of(kv, a), err);
}

template <int D, int KIND, bool INTERLEAVED>
cudaError_t launch_i(const KvView& kv, const AppendTokensArgs& a, int sms, unsigned* err, cudaStream_t st) {
  if (!a.offsets) {
    const int kv_ctas = static_cast<int>((static_cast<int64_t>(kv.batch) * kv.hkv + kThreads / (D / 16) - 1) / (kThreads / (D / 16)));
    const int64_t ctas = kv_ctas + (q_units_of(kv, a) + kWarps - 1) / kWarps;
    return launch_pdl(append_one_kernel<D, KIND, INTERLEAVED>, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), 0, st, kv, a, kv_ctas,
                      err);
  }
  constexpr int kPass = 32 / (D / 16);  // rows of a page that a warp reads at a time
  constexpr bool kBlock = KIND == HS_KV_FP8E4M3_BLOCK;
  constexpr int P = kBlock || KIND == HS_KV_FP8E4M3_G32 ? 2 : 4;
  if (kv.block <= 2 * kPass) return launch_rows<D, KIND, INTERLEAVED, 1, 2>(kv, a, sms, err, st);
  if (kv.block <= 4 * kPass) return launch_rows<D, KIND, INTERLEAVED, 1, P>(kv, a, sms, err, st);
  if constexpr (kBlock)
    if (kv.block > P * kWarps * kPass && kv_units_of(kv, a) <= static_cast<int64_t>(sms) * (threads_per_sm(KIND, 4) / kThreads))
      return launch_rows<D, KIND, INTERLEAVED, kWarps, 4>(kv, a, sms, err, st);
  return launch_rows<D, KIND, INTERLEAVED, kWarps, P>(kv, a, sms, err, st);
}

template <int D, int KIND>
cudaError_t launch_k(const KvView& kv, const AppendTokensArgs& a, int sms, unsigned* err, cudaStream_t st) {
  return a.interleaved ? launch_i<D, KIND, true>(kv, a, sms, err, st) : launch_i<D, KIND, false>(kv, a, sms, err, st);
}

template <int D>
cudaError_t launch_d(const KvView& kv, const AppendTokensArgs& a, int sms, unsigned* err, cudaStream_t st) {
  switch (kv.kv_dtype) {
    case HS_KV_F32: return launch_k<D, HS_KV_F32>(kv, a, sms, err, st);
    case HS_KV_BF16: return launch_k<D, HS_KV_BF16>(kv, a, sms, err, st);
    case HS_KV_FP8E4M3_G32: return launch_k<D, HS_KV_FP8E4M3_G32>(kv, a, sms, err, st);
    default: return launch_k<D, HS_KV_FP8E4M3_BLOCK>(kv, a, sms, err, st);
  }
}

}  // namespace

bool append_tokens_fits(const KvView& kv, const AppendTokensArgs& a) {
  return static_cast<int64_t>(kv.batch) * kv.hkv <= INT32_MAX &&
         (a.offsets ? kv_units_of(kv, a) : 0) + a.rows * ceil_div(kv.hq, kQHeads) <= INT32_MAX;
}

cudaError_t launch_append_tokens(const KvView& kv, const AppendTokensArgs& a, int sms, unsigned* err,
                                 cudaStream_t st) {
  if (kv.batch == 0 || (a.rows == 0 && !a.offsets)) return cudaSuccess;  // (offsets are checked for no rows too)
  return kv.head_dim == 128 ? launch_d<128>(kv, a, sms, err, st) : launch_d<64>(kv, a, sms, err, st);
}

}  // namespace hs
