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
// Products on the warp-level matrix instruction m16n8k16, rows of A = query heads:
//   S[head][token] = Q . C^T   bf16, a group of 32 channels (two instructions) at a time,
//     because every token's group has its own scale;
//   O[head][channel] += P . C  f16, over 16 tokens.
// Heads as rows: S lies in a lane's registers as P is wanted, so nothing is exchanged
// between lanes but the maxima.  Up to 8 heads leave half of the rows; P's second term
// goes there, which makes the two terms one instruction.
//
// Codes become operands without a conversion.  A lane loads 8 of them as a word;
// masking 4 bits out of either half of it gives two numbers n = c + 8:
//   K: as they stand, bf16 numbers below the normal ones, n 2^-133 and 16 n 2^-133, which
//     the matrix units multiply exactly (q times a power of two brings the products back
//     to size, its odd channels by 1/16); the sum starts at -8 sum q.
//   V: with the exponent of 2^10 set, f16 1024 + n and 1024 + 16 n; one two-wide
//     subtraction makes them c and 16 c.  (They are sums over the whole context, so n
//     itself would have to cancel against 8: a flat softmax over 60000 tokens would lose
//     its digits.)  V's transposition is ldmatrix's: its 16-bit units are 4 codes of a
//     token.
// The centres' products are instructions of their own: for K the row's centres times
// sum q as three bf16 terms, for V two bf16 terms of P times the record of scales and
// centres as it lies in memory.
//
// Precision: q is exact (bf16, times a power of two, which takes entries up to 2^90), S
// and all sums fp32.  P times s, in units of 2^-14 of the reference (the largest power of
// two met of s and z / 8), as two f16 terms: 22 bits, absolutely 2^-25 of the units; P
// times z as two bf16 terms, 16 bits.
#include <limits.h>

#include <atomic>

#include "attn_parts.cuh"
#include "int4.cuh"

namespace hs {
namespace {

using namespace parts;

constexpr int kStages = 3;  // tiles in a warp's ring
__host__ __device__ constexpr int teams_of(int, int nt) { return nt == 1 ? 3 : 2; }

template <int D>
struct Stage {  // byte offsets in a stage of the ring
  static constexpr int kRow = int4::row_bytes(D);
  static constexpr int kV = kTile * kRow, kRec = 2 * kTile * kRow, kRecV = kRec + kTile * 16, kBytes = kRecV + kTile * 16;
};
template <int D, int NT>
constexpr int ring_bytes() {
  return teams_of(D, NT) * kTeamWarps * kStages * Stage<D>::kBytes;
}

// Where 16-byte piece c (a group of channels) of row r of a tile lies: the reads of 8
// rows' piece c have no bank conflicts.
template <int D>
__device__ __forceinline__ uint32_t piece_at(int r, int c) {
  return D == 128 ? r * 64 + ((c ^ ((r >> 1) & 3)) << 4) : r * 32 + ((c ^ ((r >> 2) & 1)) << 4);
}

__device__ __forceinline__ void copy8(uint32_t dst, const void* src, bool live) {
  const int n = live ? 8 : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void load4(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void load4_trans(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
// d = a b + c
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1,
                                         float c0, float c2) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%11,%11};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c2));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float lower(uint32_t two) { return __uint_as_float(two << 16); }        // of two bf16
__device__ __forceinline__ float upper(uint32_t two) { return __uint_as_float(two & 0xffff0000u); }
// n (or 16 n) of two of V's codes, as f16 with 2^10 added -> c (or 16 c)
__device__ __forceinline__ uint32_t centred(uint32_t two, uint32_t minus) {
  const __half2 x = __hadd2(*reinterpret_cast<const __half2*>(&two), *reinterpret_cast<const __half2*>(&minus));
  return *reinterpret_cast<const uint32_t*>(&x);
}

template <int D, int NT>
__global__ __launch_bounds__(teams_of(D, NT) * kTeamWarps * 32, 1) void attn_int4_kernel(KvView kv, PartArgs a, unsigned* err) {
  constexpr int kTeams = teams_of(D, NT), kWarps = kTeams * kTeamWarps;
  using At = Stage<D>;
  constexpr int kGroups = D / kQuantGroup;
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
  const int g = lane >> 2, c4 = lane & 3;
  const int G = kv.group;
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
    for (int j = n.part + (slot + cut.slots - n.part % cut.slots) % cut.slots; j < n.part + n.count; j += cut.slots) {
      const int at = j / cut.slots - listed;
      if (at >= 0 && at < kListed) s_parts[tm][at] = Part{p, j - n.part, n.count, n.row};
    }
  };
  const int all_parts = number_parts(kv, a, cut, team, s_scratch[tm], note);

  uint8_t* my_ring = ring + warp * (kStages * At::kBytes);
  const uint32_t ring_addr = smem_addr(my_ring);
  // what a lane copies: piece lane % kPieces of row lane / kPieces of kRowsPer; the
  // record of row `lane`
  const uint8_t* k_piece = static_cast<const uint8_t*>(kv.k_pages) + 16 * (lane % kPieces);
  const uint8_t* v_piece = static_cast<const uint8_t*>(kv.v_pages) + 16 * (lane % kPieces);
  const uint8_t* k_recs = reinterpret_cast<const uint8_t*>(kv.k_scales);
  const uint8_t* v_recs = reinterpret_cast<const uint8_t*>(kv.v_scales);
  // what it reads: row lane % 8 of matrix lane / 8
  const int mat = lane >> 3, mr = lane & 7;

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
    const int L = kv.seq_lens[b];
    // the query's loads go out ahead of the rows'
    uint4 q_raw[NT][kGroups];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < kGroups; ++k) {
        q_raw[nt][k] = make_uint4(0u, 0u, 0u, 0u);
        if (nt * 8 + g < G)
          q_raw[nt][k] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) +
                                                              (static_cast<int64_t>(b) * kv.hq + kvh * G + nt * 8 + g) * D + 32 * k + 8 * c4));
      }
    // The warp's tiles: a run of the part.
    const int run0 = seg0 + seg_tiles * team_warp / team.warps;
    const int tiles = seg0 + seg_tiles * (team_warp + 1) / team.warps - run0;
    TileRows rows;
    rows.start(kv, a.sel + static_cast<int64_t>(part.pair) * a.capacity, kv.page_table + static_cast<int64_t>(part.pair) * kv.max_blocks, cnt,
               L, run0, tiles, lane, err);
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
#pragma unroll
      for (int i = 0; i < kTile / kRowsPer; ++i) {
        const int r = i * kRowsPer + lane / kPieces;
        const uint64_t at = static_cast<uint64_t>(__shfl_sync(0xffffffffu, row, r)) * At::kRow;
        const bool there = (live >> r) & 1u;
        copy16_if(dst + piece_at<D>(r, lane % kPieces), k_piece + at, there);
        copy16_if(dst + At::kV + piece_at<D>(r, lane % kPieces), v_piece + at, there);
      }
      const uint64_t rec = static_cast<uint64_t>(row) * (D / 8);
      if constexpr (D == 128) {
        copy16_if(dst + At::kRec + lane * 16, k_recs + rec, ok);
        copy16_if(dst + At::kRecV + lane * 16, v_recs + rec, ok);
      } else {
        copy8(dst + At::kRec + lane * 16, k_recs + rec, ok);
        copy8(dst + At::kRecV + lane * 16, v_recs + rec, ok);
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

    // ---- the query, as first operands ----
    uint32_t qa[NT][kGroups][4];  // even channels 0 4 and 2 6 of a lane's 8, then the odd ones by 1/16
    float q8[NT][kGroups];        // what the sum starts at
    uint32_t xa[NT][2];           // the groups' sums as three bf16 terms, k = term * groups + group
    float f[NT];                  // from S times the scale to a logit (log2 units)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float amax = 0.0f, sum[kGroups], x[kGroups][8];
#pragma unroll
      for (int k = 0; k < kGroups; ++k) {
        const uint32_t w[4] = {q_raw[nt][k].x, q_raw[nt][k].y, q_raw[nt][k].z, q_raw[nt][k].w};
        sum[k] = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[k][2 * i] = lower(w[i]);
          x[k][2 * i + 1] = upper(w[i]);
          amax = fmaxf(amax, fmaxf(fabsf(x[k][2 * i]), fabsf(x[k][2 * i + 1])));
          sum[k] += x[k][2 * i] + x[k][2 * i + 1];
        }
        sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], 1);
        sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], 2);
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      // times 2^e, the largest entry in [2^100, 2^101) where e is from 10 to 127
      const int e = min(max(227 - static_cast<int>(__float_as_uint(amax) >> 23), 10), 127);
      const float up = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
      f[nt] = a.scale * kLog2e * __uint_as_float(static_cast<uint32_t>(133 - e + 127) << 23);
      float t[3][kGroups];  // sum q times the logits' factor, in three terms
#pragma unroll
      for (int k = 0; k < kGroups; ++k) {
        qa[nt][k][0] = pack_bf16(x[k][0] * up, x[k][4] * up);
        qa[nt][k][1] = pack_bf16(x[k][2] * up, x[k][6] * up);
        qa[nt][k][2] = pack_bf16(x[k][1] * up * 0.0625f, x[k][5] * up * 0.0625f);
        qa[nt][k][3] = pack_bf16(x[k][3] * up * 0.0625f, x[k][7] * up * 0.0625f);
        q8[nt][k] = -sum[k] * __uint_as_float(static_cast<uint32_t>(e - 130 + 127) << 23);  // -8 2^-133 sum q 2^e
        float rest = sum[k] * (a.scale * kLog2e);
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          t[i][k] = __bfloat162float(__float2bfloat16_rn(rest));
          rest -= t[i][k];
        }
      }
      // k = 2 c4, 2 c4 + 1 and 8 more: (D = 128) terms 0 and 1 of the groups, then term 2;
      // (D = 64) the three terms, then nothing
      if constexpr (D == 128) {
        const int i = c4 >> 1;
        const float u0 = c4 & 1 ? t[i][2] : t[i][0], u1 = c4 & 1 ? t[i][3] : t[i][1];
        const float w0 = c4 & 1 ? t[2][2] : t[2][0], w1 = c4 & 1 ? t[2][3] : t[2][1];
        xa[nt][0] = pack_bf16(u0, u1);
        xa[nt][1] = c4 < 2 ? pack_bf16(w0, w1) : 0u;
      } else {
        const float u0 = c4 == 0 ? t[0][0] : c4 == 1 ? t[1][0] : t[2][0], u1 = c4 == 0 ? t[0][1] : c4 == 1 ? t[1][1] : t[2][1];
        xa[nt][0] = c4 < 3 ? pack_bf16(u0, u1) : 0u;
        xa[nt][1] = 0u;
      }
    }

    float m[NT], l[NT], base[NT];  // base: the maximum, 0 as long as there is none
    float o[kGroups][4][4];        // rows g and g + 8 (up to 8 heads: P's second term), channels 32 k + 4 (2 c4 + e) + i
    float oz[4];                   // the centres' sums: column kGroups + k of the record
    float vref = kMinRef;          // power of two, not below the V scales and centres / 8 met
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt] = -INFINITY;
      base[nt] = l[nt] = 0.0f;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      oz[e] = 0.0f;
#pragma unroll
      for (int k = 0; k < kGroups; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[k][i][e] = 0.0f;
    }

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
      const uint8_t* st = my_ring + stage * At::kBytes;
      const uint32_t st_addr = ring_addr + stage * At::kBytes;
      const uint32_t live = s_live[warp][stage];

      // ---- logits (log2 units) of 8 tokens at a time ----
      float x[NT][4][2];  // tokens 8 i + 2 c4, 8 i + 2 c4 + 1 of head g (and g + 8)
      uint32_t kw[4];     // codes of the 8 tokens' four groups, or of 16 tokens' two
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (D == 128)
          load4(st_addr + piece_at<D>(8 * i + mr, mat), kw);
        else if (i % 2 == 0)
          load4(st_addr + piece_at<D>(8 * i + 8 * (mat >> 1) + mr, mat & 1), kw);
        float s[kGroups][4], sz[4];
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
          const uint32_t v = kw[D == 128 ? k : 2 * (i % 2) + k], v8 = v >> 8;
          mma_bf16(s[k], qa[0][k][0], qa[NT - 1][k][0], qa[0][k][1], qa[NT - 1][k][1], v & 0x000f000fu, v8 & 0x000f000fu, q8[0][k],
                   q8[NT - 1][k]);
          mma_bf16(s[k], qa[0][k][2], qa[NT - 1][k][2], qa[0][k][3], qa[NT - 1][k][3], v & 0x00f000f0u, v8 & 0x00f000f0u);
        }
        const uint8_t* rec = st + At::kRec + 128 * i;
        const uint32_t z = *reinterpret_cast<const uint32_t*>(rec + 16 * g + (D == 128 ? 8 + 4 * (c4 & 1) : 4));
        mma_bf16(sz, xa[0][0], xa[NT - 1][0], xa[0][1], xa[NT - 1][1], z, z, 0.0f, 0.0f);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float sc[kGroups];
          const uint2 two = *reinterpret_cast<const uint2*>(rec + 16 * (2 * c4 + e));
          sc[0] = lower(two.x);
          sc[1] = upper(two.x);
          if constexpr (D == 128) {
            sc[2] = lower(two.y);
            sc[3] = upper(two.y);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float sum = s[0][2 * nt + e] * sc[0];
#pragma unroll
            for (int k = 1; k < kGroups; ++k) sum = fmaf(s[k][2 * nt + e], sc[k], sum);
            x[nt][i][e] = fmaf(sum, f[nt], sz[2 * nt + e]);
          }
        }
      }
      if (live != 0xffffffffu) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (!((live >> (8 * i + 2 * c4 + e)) & 1u)) {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) x[nt][i][e] = -INFINITY;
            }
      }
      bool raised = false;
      float mn[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float top = fmaxf(fmaxf(fmaxf(x[nt][0][0], x[nt][0][1]), fmaxf(x[nt][1][0], x[nt][1][1])),
                          fmaxf(fmaxf(x[nt][2][0], x[nt][2][1]), fmaxf(x[nt][3][0], x[nt][3][1])));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        mn[nt] = fmaxf(m[nt], top);
        raised |= mn[nt] > m[nt];
      }
      uint32_t vmax;
      {
        const uint4 r = *reinterpret_cast<const uint4*>(st + At::kRecV + 16 * lane);
        const auto wide = [](uint32_t p, uint32_t q) { return fmaxf(fmaxf(fabsf(lower(p)), fabsf(upper(p))), fmaxf(fabsf(lower(q)), fabsf(upper(q)))); };
        const float top = D == 128 ? fmaxf(wide(r.x, r.y), 0.125f * wide(r.z, r.w)) : fmaxf(wide(r.x, r.x), 0.125f * wide(r.y, r.y));
        vmax = __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(top, 0.0f)));  // (NaN: 0)
      }
      const uint32_t vcap = max(__float_as_uint(vref), min((vmax + 0x7fffffu) & 0x7f800000u, kMaxRef));
      if (__any_sync(0xffffffffu, raised) || vcap != __float_as_uint(vref)) {
        const float vnew = __uint_as_float(vcap);
        const float down = vref / vnew;
        vref = vnew;
        float by[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float was = m[nt] == -INFINITY ? 0.0f : exp2f(m[nt] - mn[nt]);
          l[nt] *= was;
          m[nt] = mn[nt];
          base[nt] = mn[nt] == -INFINITY ? 0.0f : mn[nt];
          by[nt] = was * down;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float y = by[(e >> 1) * (NT - 1)];
          oz[e] *= y;
#pragma unroll
          for (int k = 0; k < kGroups; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[k][i][e] *= y;
        }
      }
      const float unit = unit_over(vref);

      // ---- P, and O += P C, 16 tokens at a time ----
      uint32_t zr[4];  // records: scales in the first columns, centres behind them
      load4_trans(st_addr + At::kRecV + 16 * lane, zr);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float p[NT][4];  // tokens 16 j + 2 c4, + 1, + 8, + 9
        uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float y = exp2_fast(x[nt][2 * j + (i >> 1)][i & 1] - base[nt]);
            l[nt] += y;
            p[nt][i] = y * unit;
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            hi[nt][i] = pack_bf16(p[nt][2 * i], p[nt][2 * i + 1]);
            lo[nt][i] = pack_bf16(p[nt][2 * i] - lower(hi[nt][i]), p[nt][2 * i + 1] - upper(hi[nt][i]));
          }
        }
        if constexpr (NT == 1) {
          mma_bf16(oz, hi[0][0], lo[0][0], hi[0][1], lo[0][1], zr[2 * j], zr[2 * j + 1]);
        } else {
          mma_bf16(oz, hi[0][0], hi[NT - 1][0], hi[0][1], hi[NT - 1][1], zr[2 * j], zr[2 * j + 1]);
          mma_bf16(oz, lo[0][0], lo[NT - 1][0], lo[0][1], lo[NT - 1][1], zr[2 * j], zr[2 * j + 1]);
        }
        float sc[4][kGroups];  // the tokens' scales
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint2 two = *reinterpret_cast<const uint2*>(st + At::kRecV + 16 * (16 * j + 8 * (i >> 1) + 2 * c4 + (i & 1)));
          sc[i][0] = lower(two.x);
          sc[i][1] = upper(two.x);
          if constexpr (D == 128) {
            sc[i][2] = lower(two.y);
            sc[i][3] = upper(two.y);
          }
        }
#pragma unroll
        for (int k2 = 0; k2 < kGroups; k2 += 2) {
          uint32_t w[4];  // tokens 16 j .. + 7 and + 8 .. + 15 of groups k2 and k2 + 1
          load4_trans(st_addr + At::kV + piece_at<D>(16 * j + 8 * (mat & 1) + mr, k2 + (mat >> 1)), w);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int k = k2 + h;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const float y0 = p[nt][2 * i] * sc[2 * i][k], y1 = p[nt][2 * i + 1] * sc[2 * i + 1][k];
                hi[nt][i] = pack_half2(y0, y1);
                const float2 back = unpack_half2(hi[nt][i]);
                lo[nt][i] = pack_half2(y0 - back.x, y1 - back.y);
              }
            const uint32_t w0 = w[2 * h], w1 = w[2 * h + 1];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t mask = i & 1 ? 0x00f000f0u : 0x000f000fu;
              const uint32_t minus = i & 1 ? 0xe480e480u : 0xe408e408u;  // -1152, -1032
              const uint32_t b0 = centred(((i < 2 ? w0 : w0 >> 8) & mask) | 0x64006400u, minus);
              const uint32_t b1 = centred(((i < 2 ? w1 : w1 >> 8) & mask) | 0x64006400u, minus);
              if constexpr (NT == 1) {
                mma_f16(o[k][i], hi[0][0], lo[0][0], hi[0][1], lo[0][1], b0, b1);
              } else {
                mma_f16(o[k][i], hi[0][0], hi[NT - 1][0], hi[0][1], hi[NT - 1][1], b0, b1);
                mma_f16(o[k][i], lo[0][0], lo[NT - 1][0], lo[0][1], lo[NT - 1][1], b0, b1);
              }
            }
          }
        }
      }
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    copies_wait<0>();

    // ---- the warps' states joined ----
    team.sync();  // every warp is done with its ring: the team's rings now hold the outputs
    if (lane == 0) s_ref[warp] = vref;
    float* so = reinterpret_cast<float*>(ring + first_warp * (kStages * At::kBytes));  // [team warp][8 NT][D]
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float sum = l[nt];
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      const int h = nt * 8 + g;
      if (c4 == 0) {
        s_m[warp][h] = m[nt];
        s_l[warp][h] = sum;
      }
      // centre k is column kGroups + k: lane (kGroups + k) / 2 of the head's four
      const float z0 = NT == 1 ? oz[0] + oz[2] : oz[2 * nt], z1 = NT == 1 ? oz[1] + oz[3] : oz[2 * nt + 1];
#pragma unroll
      for (int k = 0; k < kGroups; ++k) {
        const float z = __shfl_sync(0xffffffffu, k & 1 ? z1 : z0, (lane & ~3) | ((kGroups + k) >> 1));
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float y[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            y[i] = fmaf(NT == 1 ? o[k][i][e] + o[k][i][2 + e] : o[k][i][2 * nt + e], i & 1 ? 0.0625f : 1.0f, z);
          *reinterpret_cast<float4*>(so + (team_warp * 8 * NT + h) * D + 32 * k + 4 * (2 * c4 + e)) = make_float4(y[0], y[1], y[2], y[3]);
        }
      }
    }
    team.sync();
    finish_part<D, NT>(kv, a, team, part, s_m + first_warp, s_l + first_warp, s_ref + first_warp, so, &s_last[tm]);
    team.sync();  // the rings and s_m are free again
  }
}

template <int D, int NT>
cudaError_t launch_n(const KvView& kv, const PartArgs& b, int ctas, unsigned* err, cudaStream_t st) {
  constexpr int kTeams = teams_of(D, NT);
  auto kern = attn_int4_kernel<D, NT>;
  // asked for once a device, as for the block-scaled kernel
  static std::atomic<uint64_t> allowed{0};
  int dev = 0;
  if (cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return e;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (!(allowed.load(std::memory_order_relaxed) & bit)) {
    if (cudaError_t e = allow_dynamic_smem(kern, ring_bytes<D, NT>()); e != cudaSuccess) return e;
    allowed.fetch_or(bit, std::memory_order_relaxed);
  }
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
