// Attention of one decode step over a 4-bit cache: for every token and 32 channels g
// a bf16 scale s, a bf16 centre z and codes c (int4.cuh).
//
//   logit_t = scale (sum_g s_tg (q . c_t)_g + z_tg sum_(channels of g) q)
//   out     = sum_t softmax(logit)_t (s_tg c_t + z_tg),    lse = log sum_t e^logit_t
//
// Work, its cut into parts, the joins and merges are those of the block-scaled kernel
// (attn_parts.cuh): a warp takes a run of 32-token tiles through its own ring in shared
// memory, filled by asynchronous copies.
//
// Products on the warp-level matrix instruction m16n8k16: q and codes in bf16, a group of
// 32 channels (two instructions) at a time, because every token's group has its own scale;
// P times scales and codes in f16, over 16 tokens.  Up to 8 heads are the instruction's
// narrow side, 16 its rows.
//
// Codes become operands without a conversion.  A lane loads 8 of them as a word;
// masking 4 bits out of either half of it gives two numbers n = c + 8:
//   K: as they stand, bf16 numbers below the normal ones, n 2^-133 and 16 n 2^-133, which
//     the matrix units multiply exactly (q times a power of two brings the products back
//     to size, its odd channels by 1/16); -8 sum q goes with the scale.
//   V: likewise f16 numbers, n 2^-24 and 16 n 2^-24; one two-wide subtraction makes
//     them c 2^-24 and 16 c 2^-24, exactly.  (They are sums over the whole context, so n
//     itself would have to cancel against 8: a flat softmax over 60000 tokens would lose
//     its digits.)  V's transposition is ldmatrix's: its 16-bit units are 4 codes of a
//     token.
// What scales and centres are multiplied by without the codes, -8 sum q and sum q for K,
// P for V, goes with the record as it lies in memory, in instructions of its own: three
// bf16 terms of the sums, two of P.
//
// What bounds it: the matrix, integer and fp32 pipes in turn, none of them busy half of
// the time, with instructions waiting for each other in between: 16 requests x 4 heads x
// 131072 tokens, 1.34 GB, 280 us, 0.71 of the copy rate; 64 channels 206 us for half of
// that (0.48); 16 heads 254 us for half (0.39).  32 requests x 4096 selected tokens: 29.0
// us, of which the chain of lookups before the stream and the join behind it are 7 (with
// the query asked for behind the first pages, and a slot's part found by divisions, 30.0); 12
// uneven requests of 16 heads, 64 channels: 32.0.  (Heads as rows for up to 8 heads, with
// half of the rows empty or taken by P's second term and O in twice the registers: 318.)
//
// Precision: q is exact (bf16, times a power of two, which takes entries up to 2^90), S
// and all sums fp32.  P times s, in units of 2^-13 of the reference (the largest power of
// two met of s and z / 8), as two f16 terms: 22 bits, absolutely 2^-25 of the units; P
// that z is multiplied by, in the same units, as two bf16 terms: 16 bits, absolutely 2^-134
// of the units, bf16's smallest step halved.  (With a reference of 2^126 that is 2^-21 of
// P: 12000 tokens on one CTA, most of 2^-8 and 2^-10, all of one centre, 2.3e-5 off; with
// one of 2^20 3.3e-6.)
#include <limits.h>

#include <type_traits>

#include "attn_parts.cuh"
#include "int4.cuh"

namespace hs {
namespace {

using namespace parts;

// Tiles in a warp's ring: 128 channels, two 280 us, three 282 (16 requests x 4 heads x
// 131072 tokens); 64 channels 210 and 206.
__host__ __device__ constexpr int stages_of(int head_dim) { return head_dim == 128 ? 2 : 3; }
// Logits may pass the running maximum by so much (log2 units) before the state is
// rescaled, which takes 40 products for up to 8 heads of 128 channels, 68 for 16: with
// runs of a hundred tiles every fourth tile raises a maximum, one of twenty by more than this.  P times s is in units of 2^-13 of
// the reference then, 2^15 at most.
constexpr float kMargin = 2.0f;
constexpr int kUnit4 = 13;
// Teams of a CTA (one CTA to an SM), as many as the registers allow without spilling much:
// 16 heads of 64 channels, 16 x 4 heads x 65536 tokens, 139 us (135 by now) with 12 warps, 166 with 8;
// of 128 channels 258 with 8 warps, 279 with 12.
__host__ __device__ constexpr int teams_of(int head_dim, int nt) { return head_dim == 64 || nt == 1 ? 3 : 2; }

template <int D>
struct Stage {  // byte offsets in a stage of the ring
  static constexpr int kRow = int4::row_bytes(D);
  static constexpr int kV = kTile * kRow, kRec = 2 * kTile * kRow, kRecV = kRec + kTile * 16, kBytes = kRecV + kTile * 16;
};
template <int D, int NT>
constexpr int ring_bytes() {
  return teams_of(D, NT) * kTeamWarps * stages_of(D) * Stage<D>::kBytes;
}

// Where 16-byte piece c (a group of channels) of row r of a tile lies: the reads of 8
// rows' piece c have no bank conflicts.
template <int D>
__device__ __forceinline__ uint32_t piece_at(int r, int c) {
  return D == 128 ? r * 64 + ((c ^ ((r >> 1) & 3)) << 4) : r * 32 + ((c ^ ((r >> 2) & 1)) << 4);
}

// n 2^-24 (or 16 times that) of two of V's codes, as f16 -> c 2^-24
__device__ __forceinline__ uint32_t centred(uint32_t two, uint32_t minus) {
  const __half2 x = __hadd2(*reinterpret_cast<const __half2*>(&two), *reinterpret_cast<const __half2*>(&minus));
  return *reinterpret_cast<const uint32_t*>(&x);
}

// The largest V scale, or eighth of a centre, of a tile's records, as bits (NaN: 0).
template <int D>
__device__ __forceinline__ uint32_t largest_of(const uint8_t* records, int lane) {
  const uint4 r = *reinterpret_cast<const uint4*>(records + 16 * lane);
  const auto wide = [](uint32_t p, uint32_t q) { return fmaxf(fmaxf(fabsf(lower(p)), fabsf(upper(p))), fmaxf(fabsf(lower(q)), fabsf(upper(q)))); };
  const float top = D == 128 ? fmaxf(wide(r.x, r.y), 0.125f * wide(r.z, r.w)) : fmaxf(wide(r.x, r.x), 0.125f * wide(r.y, r.y));
  return __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(top, 0.0f)));
}
// The scales of a record and the next one's, by group.
__device__ __forceinline__ void scale_pairs(const uint8_t* record, float2 (&sc)[4]) {
  const uint2 r0 = *reinterpret_cast<const uint2*>(record), r1 = *reinterpret_cast<const uint2*>(record + 16);
  sc[0] = make_float2(lower(r0.x), lower(r1.x));
  sc[1] = make_float2(upper(r0.x), upper(r1.x));
  sc[2] = make_float2(lower(r0.y), lower(r1.y));
  sc[3] = make_float2(upper(r0.y), upper(r1.y));
}
// Two f16 terms of two numbers.  MIXED: the first leaves them without being widened.
template <bool MIXED>
__device__ __forceinline__ void two_terms(float2 y, uint32_t& hi, uint32_t& lo) {
  hi = pack_half2(y.x, y.y);
  const float2 rest = MIXED ? less_f16(y, hi) : fma2(unpack_half2(hi), both(-1.0f), y);
  lo = pack_half2(rest.x, rest.y);
}
// Codes i (of the four in each half) of two tokens' 16 bits, centred, times 2^-24 (odd i: 2^-20).
__device__ __forceinline__ uint32_t centred_code(uint32_t w, int i) {
  return centred((i < 2 ? w : w >> 8) & (i & 1 ? 0x00f000f0u : 0x000f000fu), i & 1 ? 0x80808080u : 0x80088008u);
}

// Up to 8 heads: tokens as rows, heads on the instruction's narrow side.
//   S[token][head] = C . Q^T,  O^T[channel][head] += C^T . P^T
// P is transposed between the two, 16 bits at a time.
template <int D>
struct TokensInRows {
  using At = Stage<D>;
  static constexpr int kHeads = 8, kGroups = D / kQuantGroup;
  const int lane, g, c4;
  uint32_t k_at[kGroups / 2], v_at[kGroups / 2], z_at;  // what the lane reads of a tile
  uint32_t qb[kGroups][4], xb[3];
  float2 f;                 // of heads 2 c4 and + 1, as all that follows
  float2 l, m, base;        // base: the maximum, 0 as long as there is none
  float o[kGroups][2][4];   // channels 32 k + 4 g + 2 i and + 1 (rows g and g + 8; odd ones 16 times too large)
  float oz[2][4];           // row g: what column g of the records adds up to, over the first 16 tokens of each tile; row g + 8 of
                            // the second: over the others
  float vref;               // power of two, not below the V scales and centres / 8 met

  // The query's channels of the lane: asked for before the lookups of the first rows.
  struct Query {
    uint4 raw[kGroups];
    __device__ __forceinline__ Query(const KvView& kv, const PartArgs& a, int64_t head0, int lane) {
      const int g = lane >> 2, c4 = lane & 3;
#pragma unroll
      for (int k = 0; k < kGroups; ++k)
        raw[k] = g < kv.group ? __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + (head0 + g) * D + 32 * k + 8 * c4))
                              : make_uint4(0u, 0u, 0u, 0u);
    }
  };

  __device__ __forceinline__ TokensInRows(const Query& query, float scale, int this_lane)
      : lane(this_lane), g(this_lane >> 2), c4(this_lane & 3), vref(kMinRef) {
    const int mat = lane >> 3, mr = lane & 7;
#pragma unroll
    for (int k = 0; k < kGroups; k += 2) {
      k_at[k / 2] = piece_at<D>(8 * (mat & 1) + mr, k + (mat >> 1));
      v_at[k / 2] = At::kV + k_at[k / 2];
    }
    z_at = At::kRecV + 16 * (8 * (mat >> 1) + 16 * (mat & 1) + mr);  // tokens 0, 16, 8 and 24 on
    const Int4Query<kGroups> q(query.raw, scale, c4);
#pragma unroll
    for (int k = 0; k < kGroups; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) qb[k][i] = q.q[k][i];
#pragma unroll
    for (int i = 0; i < 3; ++i) xb[i] = q.terms[i];
    f = make_float2(__shfl_sync(0xffffffffu, q.factor, 8 * c4), __shfl_sync(0xffffffffu, q.factor, 8 * c4 + 4));
    l = base = both(0.0f);
    m = both(-INFINITY);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      oz[0][e] = oz[1][e] = 0.0f;
#pragma unroll
      for (int k = 0; k < kGroups; ++k) o[k][0][e] = o[k][1][e] = 0.0f;
    }
  }

  __device__ __forceinline__ void tile(const uint8_t* st, uint32_t st_addr, uint32_t live) {
    // ---- logits (log2 units), 16 tokens at a time ----
    float2 x[2][2];  // tokens 16 j + 8 e + g
    uint32_t kr[4];  // the records, 8 tokens each
    load4(st_addr + At::kRec + 16 * lane, kr);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float s[kGroups][4], add[4];
#pragma unroll
      for (int k2 = 0; k2 < kGroups; k2 += 2) {
        uint32_t w[4];  // rows g and g + 8 of group k2, then of the next
        load4(st_addr + k_at[k2 / 2] + j * (16 * At::kRow), w);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int k = k2 + h;
          const uint32_t u = w[2 * h], v = w[2 * h + 1], u8 = u >> 8, v8 = v >> 8;
          mma_bf16_0(s[k], u & 0x000f000fu, v & 0x000f000fu, u8 & 0x000f000fu, v8 & 0x000f000fu, qb[k][0], qb[k][1]);
          mma_bf16(s[k], u & 0x00f000f0u, v & 0x00f000f0u, u8 & 0x00f000f0u, v8 & 0x00f000f0u, qb[k][2], qb[k][3]);
        }
      }
      mma_bf16_0(add, kr[2 * j], kr[2 * j + 1], kr[2 * j], kr[2 * j + 1], xb[0], xb[1]);
      mma_bf16(add, kr[2 * j], kr[2 * j + 1], 0u, 0u, xb[2], 0u);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint2 two = *reinterpret_cast<const uint2*>(st + At::kRec + 16 * (16 * j + 8 * e + g));
        const float sc[4] = {lower(two.x), upper(two.x), lower(two.y), upper(two.y)};
        float2 sum = make_float2(s[0][2 * e] * sc[0], s[0][2 * e + 1] * sc[0]);
#pragma unroll
        for (int k = 1; k < kGroups; ++k) {
          sum.x = fmaf(s[k][2 * e], sc[k], sum.x);
          sum.y = fmaf(s[k][2 * e + 1], sc[k], sum.y);
        }
        x[j][e] = fma2(sum, f, make_float2(add[2 * e], add[2 * e + 1]));
      }
    }
    if (live != 0xffffffffu) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (!((live >> (8 * i + g)) & 1u)) x[i >> 1][i & 1] = both(-INFINITY);
    }
    float2 mn = make_float2(fmaxf(fmaxf(x[0][0].x, x[0][1].x), fmaxf(x[1][0].x, x[1][1].x)),
                            fmaxf(fmaxf(x[0][0].y, x[0][1].y), fmaxf(x[1][0].y, x[1][1].y)));
#pragma unroll
    for (int i = 4; i < 32; i <<= 1) {
      mn.x = fmaxf(mn.x, __shfl_xor_sync(0xffffffffu, mn.x, i));
      mn.y = fmaxf(mn.y, __shfl_xor_sync(0xffffffffu, mn.y, i));
    }
    mn.x = fmaxf(mn.x, m.x);
    mn.y = fmaxf(mn.y, m.y);
    const bool raised = mn.x > m.x + kMargin || mn.y > m.y + kMargin;
    const uint32_t vmax = largest_of<D>(st + At::kRecV, lane);
    const uint32_t vcap = max(__float_as_uint(vref), min((vmax + 0x7fffffu) & 0x7f800000u, kMaxRef));
    if (__any_sync(0xffffffffu, raised) || vcap != __float_as_uint(vref)) {
      const float vnew = __uint_as_float(vcap), down = vref / vnew;
      vref = vnew;
      const float2 was = make_float2(m.x == -INFINITY ? 0.0f : exp2f(m.x - mn.x), m.y == -INFINITY ? 0.0f : exp2f(m.y - mn.y));
      l = mul2(l, was);
      m = mn;
      base = make_float2(mn.x == -INFINITY ? 0.0f : mn.x, mn.y == -INFINITY ? 0.0f : mn.y);
      const float2 by = mul2(was, both(down));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float y = e & 1 ? by.y : by.x;
        oz[0][e] *= y;
        oz[1][e] *= y;
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
          o[k][0][e] *= y;
          o[k][1][e] *= y;
        }
      }
    }
    const float unit = unit_over(vref) * (1.0f / (1 << (kUnit - kUnit4)));

    // ---- P, and O^T += C^T P^T, 16 tokens at a time ----
    uint32_t zr[4];  // the records' columns: scales, then centres
    load4_trans(st_addr + z_at, zr);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float2 p[2];  // of head g: tokens 16 j + 8 e + 2 c4 and + 1
      uint32_t hi[2], lo[2];
      float2 sc[2][4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float2 y = add2(x[j][e], make_float2(-base.x, -base.y));
        const float2 w = make_float2(exp2_fast(y.x), exp2_fast(y.y));
        l = add2(l, w);
        const float2 in = mul2(w, both(unit));
        const uint32_t a = __float_as_uint(in.x), b = __float_as_uint(in.y);
        const uint32_t up = transpose8x8(__byte_perm(a, b, 0x7632)), down = transpose8x8(__byte_perm(a, b, 0x5410));
        p[e] = make_float2(__uint_as_float(__byte_perm(down, up, 0x5410)), __uint_as_float(__byte_perm(down, up, 0x7632)));
        hi[e] = pack_bf16(p[e].x, p[e].y);
        lo[e] = pack_bf16(p[e].x - lower(hi[e]), p[e].y - upper(hi[e]));
        scale_pairs(st + At::kRecV + 32 * c4 + 16 * (16 * j + 8 * e), sc[e]);
      }
      mma_bf16(oz[j], zr[0], zr[1], zr[2], zr[3], hi[0], hi[1]);
      mma_bf16(oz[j], zr[0], zr[1], zr[2], zr[3], lo[0], lo[1]);
#pragma unroll
      for (int k2 = 0; k2 < kGroups; k2 += 2) {
        uint32_t w[4];  // tokens 16 j .. + 7 and + 8 .. + 15 of groups k2 and k2 + 1
        load4_trans(st_addr + v_at[k2 / 2] + j * (16 * At::kRow), w);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int k = k2 + h;
#pragma unroll
          for (int e = 0; e < 2; ++e) two_terms<false>(mul2(p[e], sc[e][k]), hi[e], lo[e]);
          const uint32_t w0 = w[2 * h], w1 = w[2 * h + 1];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t a0 = centred_code(w0, 2 * i), a1 = centred_code(w0, 2 * i + 1);
            const uint32_t a2 = centred_code(w1, 2 * i), a3 = centred_code(w1, 2 * i + 1);
            mma_f16(o[k][i], a0, a1, a2, a3, hi[0], hi[1]);
            mma_f16(o[k][i], a0, a1, a2, a3, lo[0], lo[1]);
          }
        }
      }
    }
  }

  // The warp's state: outputs in units of 2^-kUnit of the reference.
  __device__ __forceinline__ void state(float* so, float* s_m, float* s_l, float* s_ref) const {
    float2 sum = l;
#pragma unroll
    for (int i = 4; i < 32; i <<= 1) {
      sum.x += __shfl_xor_sync(0xffffffffu, sum.x, i);
      sum.y += __shfl_xor_sync(0xffffffffu, sum.y, i);
    }
    if (lane == 0) *s_ref = vref;
    if (g == 0) {
      s_m[2 * c4] = m.x;
      s_m[2 * c4 + 1] = m.y;
      s_l[2 * c4] = sum.x;
      s_l[2 * c4 + 1] = sum.y;
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float col = oz[0][e] + oz[1][2 + e];
#pragma unroll
      for (int k = 0; k < kGroups; ++k) {
        const float z = __shfl_sync(0xffffffffu, col, 4 * (kGroups + k) + c4);  // centre k is column kGroups + k
        constexpr float kBack = static_cast<float>(1 << (kUnit - kUnit4));
        *reinterpret_cast<float4*>(so + (2 * c4 + e) * D + 32 * k + 4 * g) =
            make_float4(fmaf(o[k][0][e], 16777216.0f, z) * kBack, fmaf(o[k][0][2 + e], 1048576.0f, z) * kBack,
                        fmaf(o[k][1][e], 16777216.0f, z) * kBack, fmaf(o[k][1][2 + e], 1048576.0f, z) * kBack);
      }
    }
  }
};

// 16 heads: heads as rows.
//   S[head][token] = Q . C^T,  O[head][channel] += P . C
// S lies in a lane's registers as P is wanted, and nothing but the maxima is exchanged
// between lanes.
template <int D>
struct HeadsInRows {
  using At = Stage<D>;
  static constexpr int kHeads = 16, kGroups = D / kQuantGroup;
  const int lane, g, c4;
  uint32_t k_at, v_at[kGroups / 2];  // what the lane reads of a tile
  uint32_t qa[2][kGroups][4], xa[2][3];
  float f[2];                // of heads g and g + 8, as all that follows
  float2 l[2];
  float m[2], base[2];       // base: the maximum, 0 as long as there is none
  float o[kGroups][4][4];    // channels 32 k + 4 (2 c4 + e) + i (odd i 16 times too large)
  float oz[4];               // what columns 2 c4 and + 1 of the records add up to
  float vref;                // power of two, not below the V scales and centres / 8 met

  struct Query {  // as above, of heads g and g + 8
    uint4 raw[2][kGroups];
    __device__ __forceinline__ Query(const KvView& kv, const PartArgs& a, int64_t head0, int lane) {
      const int g = lane >> 2, c4 = lane & 3;
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int k = 0; k < kGroups; ++k)
          raw[nt][k] = nt * 8 + g < kv.group ? __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) +
                                                                                   (head0 + nt * 8 + g) * D + 32 * k + 8 * c4))
                                             : make_uint4(0u, 0u, 0u, 0u);
    }
  };

  __device__ __forceinline__ HeadsInRows(const Query& query, float scale, int this_lane)
      : lane(this_lane), g(this_lane >> 2), c4(this_lane & 3), vref(kMinRef) {
    const int mat = lane >> 3, mr = lane & 7;
    k_at = D == 128 ? piece_at<D>(mr, mat) : piece_at<D>(8 * (mat >> 1) + mr, mat & 1);  // (every 8th row is permuted alike)
#pragma unroll
    for (int k = 0; k < kGroups; k += 2) v_at[k / 2] = At::kV + piece_at<D>(8 * (mat & 1) + mr, k + (mat >> 1));
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      const Int4Query<kGroups> q(query.raw[nt], scale, c4);
#pragma unroll
      for (int k = 0; k < kGroups; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) qa[nt][k][i] = q.q[k][i];
#pragma unroll
      for (int i = 0; i < 3; ++i) xa[nt][i] = q.terms[i];
      f[nt] = q.factor;
      l[nt] = both(0.0f);
      m[nt] = -INFINITY;
      base[nt] = 0.0f;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      oz[e] = 0.0f;
#pragma unroll
      for (int k = 0; k < kGroups; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[k][i][e] = 0.0f;
    }
  }

  __device__ __forceinline__ void tile(const uint8_t* st, uint32_t st_addr, uint32_t live) {
    // ---- logits (log2 units) of 8 tokens at a time ----
    float2 x[2][4];  // tokens 8 i + 2 c4, 8 i + 2 c4 + 1
    uint32_t kw[4];  // codes of the 8 tokens' four groups, or of 16 tokens' two
    uint32_t kr[4];  // the records, 8 tokens each
    load4(st_addr + At::kRec + 16 * lane, kr);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (D == 128 || i % 2 == 0) load4(st_addr + k_at + i * (8 * At::kRow), kw);
      float s[kGroups][4], sz[4];
#pragma unroll
      for (int k = 0; k < kGroups; ++k) {
        const uint32_t v = kw[D == 128 ? k : 2 * (i % 2) + k], v8 = v >> 8;
        mma_bf16_0(s[k], qa[0][k][0], qa[1][k][0], qa[0][k][1], qa[1][k][1], v & 0x000f000fu, v8 & 0x000f000fu);
        mma_bf16(s[k], qa[0][k][2], qa[1][k][2], qa[0][k][3], qa[1][k][3], v & 0x00f000f0u, v8 & 0x00f000f0u);
      }
      mma_bf16_0(sz, xa[0][0], xa[1][0], xa[0][1], xa[1][1], kr[i], kr[i]);
      mma_bf16(sz, xa[0][2], xa[1][2], 0u, 0u, kr[i], kr[i]);
      float2 sc[4];
      scale_pairs(st + At::kRec + 32 * c4 + 128 * i, sc);
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        float2 sum = mul2(make_float2(s[0][2 * nt], s[0][2 * nt + 1]), sc[0]);
#pragma unroll
        for (int k = 1; k < kGroups; ++k) sum = fma2(make_float2(s[k][2 * nt], s[k][2 * nt + 1]), sc[k], sum);
        x[nt][i] = fma2(sum, both(f[nt]), make_float2(sz[2 * nt], sz[2 * nt + 1]));
      }
    }
    if (live != 0xffffffffu) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          if (!((live >> (8 * i + 2 * c4)) & 1u)) x[nt][i].x = -INFINITY;
          if (!((live >> (8 * i + 2 * c4 + 1)) & 1u)) x[nt][i].y = -INFINITY;
        }
    }
    bool raised = false;
    float mn[2];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      float top = fmaxf(fmaxf(fmaxf(x[nt][0].x, x[nt][0].y), fmaxf(x[nt][1].x, x[nt][1].y)),
                        fmaxf(fmaxf(x[nt][2].x, x[nt][2].y), fmaxf(x[nt][3].x, x[nt][3].y)));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      mn[nt] = fmaxf(m[nt], top);
      raised |= mn[nt] > m[nt] + kMargin;
    }
    const uint32_t vmax = largest_of<D>(st + At::kRecV, lane);
    const uint32_t vcap = max(__float_as_uint(vref), min((vmax + 0x7fffffu) & 0x7f800000u, kMaxRef));
    if (__any_sync(0xffffffffu, raised) || vcap != __float_as_uint(vref)) {
      const float vnew = __uint_as_float(vcap), down = vref / vnew;
      vref = vnew;
      float by[2];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const float was = m[nt] == -INFINITY ? 0.0f : exp2f(m[nt] - mn[nt]);
        l[nt] = mul2(l[nt], both(was));
        m[nt] = mn[nt];
        base[nt] = mn[nt] == -INFINITY ? 0.0f : mn[nt];
        by[nt] = was * down;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        oz[e] *= by[e >> 1];
#pragma unroll
        for (int k = 0; k < kGroups; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[k][i][e] *= by[e >> 1];
      }
    }
    const float unit = unit_over(vref) * (1.0f / (1 << (kUnit - kUnit4)));

    // ---- P, and O += P C, 16 tokens at a time ----
    uint32_t zr[4];  // the records' columns: scales, then centres
    load4_trans(st_addr + At::kRecV + 16 * lane, zr);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float2 p[2][2];  // tokens 16 j + 2 c4 and + 1, 8 more
      uint32_t hi[2][2], lo[2][2];
      float2 sc[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const float2 y = add2(x[nt][2 * j + i], both(-base[nt]));
          p[nt][i] = make_float2(exp2_fast(y.x), exp2_fast(y.y));
          l[nt] = add2(l[nt], p[nt][i]);
          p[nt][i] = mul2(p[nt][i], both(unit));
          hi[nt][i] = pack_bf16(p[nt][i].x, p[nt][i].y);
          const float2 rest = less_bf16(p[nt][i], hi[nt][i]);
          lo[nt][i] = pack_bf16(rest.x, rest.y);
        }
        scale_pairs(st + At::kRecV + 32 * c4 + 16 * (16 * j + 8 * i), sc[i]);
      }
      mma_bf16(oz, hi[0][0], hi[1][0], hi[0][1], hi[1][1], zr[2 * j], zr[2 * j + 1]);
      mma_bf16(oz, lo[0][0], lo[1][0], lo[0][1], lo[1][1], zr[2 * j], zr[2 * j + 1]);
#pragma unroll
      for (int k2 = 0; k2 < kGroups; k2 += 2) {
        uint32_t w[4];  // tokens 16 j .. + 7 and + 8 .. + 15 of groups k2 and k2 + 1
        load4_trans(st_addr + v_at[k2 / 2] + j * (16 * At::kRow), w);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int k = k2 + h;
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) two_terms<true>(mul2(p[nt][i], sc[i][k]), hi[nt][i], lo[nt][i]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t b0 = centred_code(w[2 * h], i), b1 = centred_code(w[2 * h + 1], i);
            mma_f16(o[k][i], hi[0][0], hi[1][0], hi[0][1], hi[1][1], b0, b1);
            mma_f16(o[k][i], lo[0][0], lo[1][0], lo[0][1], lo[1][1], b0, b1);
          }
        }
      }
    }
  }

  // The warp's state: outputs in units of 2^-kUnit of the reference.
  __device__ __forceinline__ void state(float* so, float* s_m, float* s_l, float* s_ref) const {
    if (lane == 0) *s_ref = vref;
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      float sum = l[nt].x + l[nt].y;
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      const int h = nt * 8 + g;
      if (c4 == 0) {
        s_m[h] = m[nt];
        s_l[h] = sum;
      }
#pragma unroll
      for (int k = 0; k < kGroups; ++k) {
        // centre k is column kGroups + k: lane (kGroups + k) / 2 of the head's four
        const float z = __shfl_sync(0xffffffffu, k & 1 ? oz[2 * nt + 1] : oz[2 * nt], (lane & ~3) | ((kGroups + k) >> 1));
        constexpr float kBack = static_cast<float>(1 << (kUnit - kUnit4));
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int at = 2 * nt + e;
          *reinterpret_cast<float4*>(so + h * D + 32 * k + 4 * (2 * c4 + e)) =
              make_float4(fmaf(o[k][0][at], 16777216.0f, z) * kBack, fmaf(o[k][1][at], 1048576.0f, z) * kBack,
                          fmaf(o[k][2][at], 16777216.0f, z) * kBack, fmaf(o[k][3][at], 1048576.0f, z) * kBack);
        }
      }
    }
  }
};

template <int D, int NT>
__global__ __launch_bounds__(teams_of(D, NT) * kTeamWarps * 32, 1) void attn_int4_kernel(KvView kv, PartArgs a, unsigned* err) {
  constexpr int kTeams = teams_of(D, NT), kWarps = kTeams * kTeamWarps;
  using At = Stage<D>;
  constexpr int kStages = stages_of(D);
  using Math = std::conditional_t<NT == 1, TokensInRows<D>, HeadsInRows<D>>;
  // a team's rings hold the outputs of its warps, and the weights of a pair's parts where it merges them
  constexpr int kRings = kTeamWarps * kStages * At::kBytes, kMostCtas = 160;
  static_assert(kTeamWarps * 8 * NT * D * 4 <= kRings && 8 * NT * (kMostCtas * kTeams + 2) * 4 + 16 <= kRings);
  constexpr int kPieces = At::kRow / 16;  // 16-byte pieces of a row, a group of channels each
  constexpr int kRowsPer = 32 / kPieces;  // rows one copy instruction of a warp covers
  extern __shared__ __align__(1024) uint8_t ring[];
  __shared__ uint32_t s_live[kWarps][kStages];
  __shared__ float s_m[kWarps][8 * NT], s_l[kWarps][8 * NT], s_ref[kWarps];
  __shared__ Scratch s_scratch[kTeams];
  __shared__ Part s_parts[kTeams][kListed];
  __shared__ int s_last[kTeams], s_empty;
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) s_empty = 0;
  __syncthreads();
  const int ctas = gridDim.x;

  const Team cta{tid, kWarps, 0};
  const Cut cut = choose_cut(kv, a, ctas, kTeams, cta, s_scratch[0], [&](int p, int count) {
    if (p % ctas == static_cast<int>(blockIdx.x)) {  // the CTA that answers for the pair's count
      if (count == 0) s_empty = 1;
      if (a.sel_count[p] > a.capacity) set_error(err, HS_EBIT_CAPACITY);
    }
  });
  if (s_empty) answer_empty<D>(kv, a, tid, kWarps * 32);
  const int tm = cut.joint ? 0 : warp / kTeamWarps, first_warp = tm * kTeamWarps, team_warp = warp - first_warp;
  const Team team = cut.joint ? cta : Team{tid - tm * kTeamWarps * 32, kTeamWarps, 1 + tm};
  const int slot = tm * ctas + blockIdx.x;  // (the first slots are on different SMs)
  int listed = 0;                           // parts of this team noted so far
  const auto note = [&](int p, const Pairs& n) {
    // this team's parts among the pair's, the next kListed of them
    if (n.part + n.count <= cut.slots) {  // no slot has two: without the divisions
      if (slot >= n.part && slot < n.part + n.count && listed == 0) s_parts[tm][0] = Part{p, slot - n.part, n.count, n.row};
      return;
    }
    for (int j = n.part + (slot + cut.slots - n.part % cut.slots) % cut.slots; j < n.part + n.count; j += cut.slots) {
      const int at = j / cut.slots - listed;
      if (at >= 0 && at < kListed) s_parts[tm][at] = Part{p, j - n.part, n.count, n.row};
    }
  };
  const int all_parts = number_parts(kv, a, cut, team, s_scratch[tm], note);

  uint8_t* my_ring = ring + warp * (kStages * At::kBytes);
  const uint32_t ring_addr = smem_addr(my_ring);
  // what a lane copies: 16 bytes of a row's codes (kPieces lanes to a row), and the record of row `lane`
  const bool together = (kv.block & 31) == 0;  // tiles lie within a page
  const uint8_t* k_codes = static_cast<const uint8_t*>(kv.k_pages) + 16 * lane;
  const uint8_t* v_codes = static_cast<const uint8_t*>(kv.v_pages) + 16 * lane;
  const uint8_t* k_recs = reinterpret_cast<const uint8_t*>(kv.k_scales);
  const uint8_t* v_recs = reinterpret_cast<const uint8_t*>(kv.v_scales);

  const int my_parts = (all_parts - slot + cut.slots - 1) / cut.slots;
  for (int n_part = 0; n_part < my_parts; ++n_part) {
    if (n_part == listed + kListed) {
      listed = n_part;
      number_parts(kv, a, cut, team, s_scratch[tm], note);
    }
    // ---- the part: seg_tiles tiles of the pair from seg0 on ----
    const Part part = s_parts[tm][n_part - listed];
    const int cnt = pair_count(a, part.pair);
    const int pair_tiles = tiles_of(kv, cnt), each = pair_tiles / part.count, more = pair_tiles - each * part.count;
    const int seg0 = part.index * each + min(part.index, more), seg_tiles = each + (part.index < more ? 1 : 0);
    const int b = part.pair / kv.hkv, kvh = part.pair - b * kv.hkv;
    // The warp's tiles: a run of the part.
    const int run0 = seg0 + seg_tiles * team_warp / team.warps;
    const int tiles = seg0 + seg_tiles * (team_warp + 1) / team.warps - run0;
    const typename Math::Query query(kv, a, static_cast<int64_t>(b) * kv.hq + kvh * kv.group, lane);
    TileRows<PartArgs> rows(kv, a, part.pair, cnt, kv.seq_lens[b], run0, tiles, lane, err);
    if constexpr (D == 64) {  // the empty halves of the records
#pragma unroll
      for (int i = 0; i < kStages; ++i) {
        *reinterpret_cast<uint2*>(my_ring + i * At::kBytes + At::kRec + lane * 16 + 8) = make_uint2(0u, 0u);
        *reinterpret_cast<uint2*>(my_ring + i * At::kBytes + At::kRecV + lane * 16 + 8) = make_uint2(0u, 0u);
      }
    }
    int stage_in = 0;
    const auto issue = [&]() {  // the copies of the next tile; rows that are not there are zeros
      uint32_t row;
      const bool ok = rows.next(row);
      const uint32_t live = __ballot_sync(0xffffffffu, ok);
      const uint32_t dst = ring_addr + stage_in * At::kBytes;
      const uint32_t my = dst + piece_at<D>(lane / kPieces, lane % kPieces);  // (the same for every kRowsPer-th row)
      if (live == 0xffffffffu && together) {  // 32 rows that lie together: one address and constants
        const uint64_t first = __shfl_sync(0xffffffffu, row, 0);
        const uint8_t* k = k_codes + first * At::kRow;
        const uint8_t* v = v_codes + first * At::kRow;
#pragma unroll
        for (int i = 0; i < kTile / kRowsPer; ++i) {
          copy16(my + i * (kRowsPer * At::kRow), k + i * (kRowsPer * At::kRow));
          copy16(my + i * (kRowsPer * At::kRow) + At::kV, v + i * (kRowsPer * At::kRow));
        }
        if constexpr (D == 128) {
          copy16(dst + At::kRec + lane * 16, k_recs + static_cast<uint64_t>(row) * 16);
          copy16(dst + At::kRecV + lane * 16, v_recs + static_cast<uint64_t>(row) * 16);
        } else {
          copy8(dst + At::kRec + lane * 16, k_recs + static_cast<uint64_t>(row) * 8, true);
          copy8(dst + At::kRecV + lane * 16, v_recs + static_cast<uint64_t>(row) * 8, true);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kTile / kRowsPer; ++i) {
          const int r = i * kRowsPer + lane / kPieces;
          const uint64_t at = static_cast<uint64_t>(__shfl_sync(0xffffffffu, row, r)) * At::kRow + 16 * (lane % kPieces);
          const bool there = (live >> r) & 1u;
          copy16_if(my + i * (kRowsPer * At::kRow), static_cast<const uint8_t*>(kv.k_pages) + at, there);
          copy16_if(my + i * (kRowsPer * At::kRow) + At::kV, static_cast<const uint8_t*>(kv.v_pages) + at, there);
        }
        const uint64_t rec = static_cast<uint64_t>(row) * (D / 8);
        if constexpr (D == 128) {
          copy16_if(dst + At::kRec + lane * 16, k_recs + rec, ok);
          copy16_if(dst + At::kRecV + lane * 16, v_recs + rec, ok);
        } else {
          copy8(dst + At::kRec + lane * 16, k_recs + rec, ok);
          copy8(dst + At::kRecV + lane * 16, v_recs + rec, ok);
        }
      }
      if (lane == 0) s_live[warp][stage_in] = live;
      stage_in = stage_in + 1 == kStages ? 0 : stage_in + 1;
    };
    int issued = 0;
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
      if (issued < tiles) {
        issue();
        ++issued;
      }
      copies_commit();
    }

    Math math(query, a.scale, lane);
    int stage = 0;
    for (int n = 0; n < tiles; ++n) {
      __syncwarp();  // the stage about to be filled has been read by every lane
      if (issued < tiles) {
        issue();
        ++issued;
      }
      copies_commit();
      copies_wait<kStages - 1>();
      __syncwarp();
      math.tile(my_ring + stage * At::kBytes, ring_addr + stage * At::kBytes, s_live[warp][stage]);
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    copies_wait<0>();

    // ---- the warps' states joined ----
    team.sync();  // every warp is done with its ring: the team's rings now hold the outputs
    float* so = reinterpret_cast<float*>(ring + first_warp * (kStages * At::kBytes));  // [team warp][heads][D]
    math.state(so + team_warp * Math::kHeads * D, s_m[warp], s_l[warp], &s_ref[warp]);
    team.sync();
    finish_part<D, NT>(kv, a, team, part, s_m + first_warp, s_l + first_warp, s_ref + first_warp, so, &s_last[tm]);
    team.sync();  // the rings and s_m are free again
  }
}

template <int D, int NT>
cudaError_t launch_n(const KvView& kv, const PartArgs& b, int ctas, unsigned* err, cudaStream_t st) {
  constexpr int kTeams = teams_of(D, NT);
  auto kern = attn_int4_kernel<D, NT>;
  static std::atomic<uint64_t> allowed{0};
  if (cudaError_t e = allow_dynamic_smem_once(allowed, kern, ring_bytes<D, NT>()); e != cudaSuccess) return e;
  cudaError_t e = launch_pdl(kern, dim3(ctas), dim3(kTeams * kTeamWarps * 32), (ring_bytes<D, NT>()), st, kv, b, err);
  if (e != cudaSuccess || b.counters) return e;
  const size_t smem = (static_cast<size_t>(ctas * kTeams + 2) * kv.group + 4 + static_cast<size_t>(kTeams - 1) * kv.group * D) * sizeof(float);
  auto merge = merge_parts_kernel<D, NT, kTeams>;
  if ((e = allow_dynamic_smem(merge, smem)) != cudaSuccess) return e;
  return launch_pdl(merge, dim3(kv.batch * kv.hkv), dim3(kTeams * kTeamWarps * 32), smem, st, kv, b, ctas);
}

}  // namespace

int int4_attn_rows(int ctas, int head_dim, int group) { return 2 * ctas * teams_of(head_dim, group <= 8 ? 1 : 2); }

cudaError_t launch_int4_attn(const KvView& kv, const AttnArgs& a, unsigned* err, cudaStream_t st) {
  if (kv.batch == 0) return cudaSuccess;
  PartArgs b;
  b.q = a.q;
  b.sel = a.sel;
  b.sel_count = a.sel_count;
  b.out = a.out;
  b.lse = a.lse;
  b.ws_o = a.ws_o;
  b.ws_lse = a.ws_lse;
  b.counters = a.counters;
  b.capacity = a.capacity;
  b.out_f32 = a.out_is_fp32;
  b.scale = a.scale;
  if (kv.head_dim == 128)
    return kv.group <= 8 ? launch_n<128, 1>(kv, b, a.sms, err, st) : launch_n<128, 2>(kv, b, a.sms, err, st);
  return kv.group <= 8 ? launch_n<64, 1>(kv, b, a.sms, err, st) : launch_n<64, 2>(kv, b, a.sms, err, st);
}

}  // namespace hs
