// Attention of one decode step over a block-scaled e4m3 cache: one fp32 scale
// per page (a block of tokens of one kv head) for K and one for V.
//
//   s_t = (q . kcode_t) * kscale * scale            (kscale, vscale: of t's page)
//   out = sum_t softmax(s)_t * vscale * vcode_t,    lse = log sum_t e^(s_t)
//
// Both scales leave the products: kscale multiplies the finished logit of a
// token, vscale its probability, so the codes enter the matrix units as they
// are (as f16, which holds every e4m3 number exactly).
//
// Work: the 32-token tiles of every (request, kv head)'s selection are laid end
// to end (from the actual counts, summed by every CTA) and cut into equal
// ranges, one per CTA; a range that ends inside a pair leaves a partial result,
// and the CTA that arrives last at the pair merges them in range order (the
// same result whichever CTA that is).  The warps of a CTA take the tiles of a
// segment in turn, each with its own running maximum, sum and output, its own
// ring of tiles in shared memory filled by asynchronous 16-byte copies, and no
// barrier with the others until the segment ends.
//
// Products on the warp-level matrix instruction m16n8k16 (f16 in, fp32 sums):
//   S[token][head] = K . Q^T: 16 tokens by 8 heads, so that the group of query
//     heads that shares the kv head fills the instruction's narrow side;
//   O^T[channel][head] += V^T . P^T: 16 channels by 8 heads over 16 tokens.
// Order of the contracted channels and of the output's channels is free, so a
// lane's operands are whole 16-byte pieces of a row as it lies in memory; V's
// transposition is one byte permutation per two operands.  Rows lie in shared
// memory with their 16-byte pieces XOR-permuted, so that neither reading order
// has bank conflicts.
//
// Precision: q times a power of two per head (largest entry into [128, 256)) is
// exact in f16 for entries within 2^-21 of the largest, and absolutely within
// 2^-33 of it below.  P * vscale, in units of 2^-14 times the largest V scale
// met so far (a power of two), enters as two f16 terms (22 bits).  Sums,
// maxima and outputs are fp32.
#include "hs_internal.h"

namespace hs {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kCtasPerSm = 2;
constexpr int kTile = 32;       // tokens a warp handles at a time
constexpr int kStages = 3;      // tiles in a warp's ring
constexpr int kMinTiles = 4;    // tiles of a range at least: one per warp
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMinRef = 7.888609052210118e-31f;  // 2^-100
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// 16 bytes to shared memory; zeros, and nothing read, unless `live`
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool live) {
  const int n = live ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool live) {
  const int n = live ? 4 : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
// two e4m3 codes (the low or the high half of w) to two f16, exactly
__device__ __forceinline__ uint32_t half2_of(uint16_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3);
  return static_cast<uint32_t>(h.x) | (static_cast<uint32_t>(h.y) << 16);
}
__device__ __forceinline__ uint32_t lo2(uint32_t w) { return half2_of(static_cast<uint16_t>(w)); }
__device__ __forceinline__ uint32_t hi2(uint32_t w) { return half2_of(static_cast<uint16_t>(w >> 16)); }
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_half2(uint32_t w) { return __half22float2(*reinterpret_cast<__half2*>(&w)); }

// Where 16-byte piece c of row r (of a tile) lies.
//   128-byte rows: piece c ^ (r mod 8).
//   64-byte rows: two rows share a 128-byte line; its 8 pieces are permuted by
//   twice the line's number mod 4.
template <int D>
__device__ __forceinline__ uint32_t piece_at(int r, int c) {
  if constexpr (D == 128)
    return static_cast<uint32_t>(r * 128 + ((c ^ (r & 7)) << 4));
  else
    return static_cast<uint32_t>((r >> 1) * 128 + (((((r & 1) << 2) | c) ^ (((r >> 1) & 3) << 1)) << 4));
}
// Token (of 16) that row i of the S product holds: the reading order without
// bank conflicts.
template <int D>
__device__ __forceinline__ int token_of(int i) {
  return (D == 128 && (i & 1)) ? (i ^ 4) : i;
}

struct BlockArgs {
  const void* q;
  const int32_t* sel;
  const int32_t* sel_count;
  void* out;
  float* lse;
  float* ws_o;
  float* ws_lse;
  uint32_t* counters;  // nullable
  int32_t capacity;
  int32_t out_f32;
  float scale;
};

// Tiles of pair p's selection.
__device__ __forceinline__ int pair_count(const KvView& kv, const BlockArgs& a, int64_t p) {
  const int c = __ldg(a.sel_count + p);
  return min(max(c, 0), a.capacity);
}
__device__ __forceinline__ int64_t tiles_of(const KvView& kv, int count) {
  return (static_cast<int64_t>(count) * kv.block + kTile - 1) / kTile;
}

// Lays the pairs' tiles end to end.  Every thread of the CTA calls it with the
// same `at`; afterwards *pair / *start are the pair that holds tile `at` and its
// first tile, and the total is returned.  `each(p, count)` sees every pair once.
struct Scan {
  int64_t sums[kWarps];
  int64_t start;
  int pair;
};
template <typename F>
__device__ int64_t sum_tiles(const KvView& kv, const BlockArgs& a, Scan& sc, F&& begin, int* pair, int64_t* start) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int pairs = kv.batch * kv.hkv, per = (pairs + kThreads - 1) / kThreads;
  const int p0 = min(pairs, tid * per), p1 = min(pairs, p0 + per);
  int64_t mine = 0;
  for (int p = p0; p < p1; ++p) mine += tiles_of(kv, pair_count(kv, a, p));
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) sc.sums[warp] = incl;
  __syncthreads();
  int64_t total = 0, before = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w == warp) before = total;
    total += sc.sums[w];
  }
  const int64_t at = begin(total);
  int64_t t = before + incl - mine;
  if (at >= t && at < t + mine)
    for (int p = p0; p < p1; ++p) {
      const int64_t n = tiles_of(kv, pair_count(kv, a, p));
      if (at < t + n) {
        sc.pair = p;
        sc.start = t;
        break;
      }
      t += n;
    }
  __syncthreads();
  *pair = sc.pair;
  *start = sc.start;
  return total;
}

__device__ __forceinline__ int64_t range_length(int64_t total, int ctas) {
  const int64_t per = (total + ctas - 1) / ctas;
  return per > kMinTiles ? per : kMinTiles;
}

__device__ __forceinline__ void store_out(const BlockArgs& a, int64_t at, float4 v) {
  if (a.out_f32) {
    reinterpret_cast<float4*>(a.out)[at / 4] = v;
  } else {
    const __nv_bfloat162 x = __floats2bfloat162_rn(v.x, v.y), y = __floats2bfloat162_rn(v.z, v.w);
    reinterpret_cast<uint2*>(a.out)[at / 4] =
        make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
  }
}

// Joins the partial results of a pair (ranges c0 .. c1, in that order) into
// out / lse.  Range c's partial of the pair is row 2c when the pair was already
// under way at the range's start or begins there, else row 2c + 1.
template <int D>
__device__ void merge_pair(const KvView& kv, const BlockArgs& a, int64_t pair, int64_t start, int64_t per, int c0, int c1) {
  const int G = kv.group;
  const int first_row = 2 * c0 + (static_cast<int64_t>(c0) * per >= start ? 0 : 1);
  const int64_t b = pair / kv.hkv, kvh = pair - b * kv.hkv;
  for (int idx = threadIdx.x; idx < G * (D / 4); idx += kThreads) {
    const int h = idx / (D / 4), d = (idx - h * (D / 4)) * 4;
    float M = -INFINITY;
    for (int c = c0; c <= c1; ++c) M = fmaxf(M, __ldcg(a.ws_lse + static_cast<int64_t>(c == c0 ? first_row : 2 * c) * G + h));
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float tot = 0.0f;
    if (M != -INFINITY) {
#pragma unroll 4
      for (int c = c0; c <= c1; ++c) {
        const int64_t row = static_cast<int64_t>(c == c0 ? first_row : 2 * c) * G + h;
        const float w = expf(__ldcg(a.ws_lse + row) - M);
        const float4 v = __ldcg(reinterpret_cast<const float4*>(a.ws_o + row * D + d));
        tot += w;
        acc.x = fmaf(w, v.x, acc.x);
        acc.y = fmaf(w, v.y, acc.y);
        acc.z = fmaf(w, v.z, acc.z);
        acc.w = fmaf(w, v.w, acc.w);
      }
      acc = make_float4(acc.x / tot, acc.y / tot, acc.z / tot, acc.w / tot);
    }
    const int64_t row = b * kv.hq + kvh * G + h;
    store_out(a, row * D + d, acc);
    if (d == 0 && a.lse) a.lse[row] = M == -INFINITY ? M : M + logf(tot);
  }
}

template <int D>
constexpr int ring_bytes() {
  return kWarps * kStages * 2 * kTile * D;
}

template <int D, int NT>
__global__ __launch_bounds__(kThreads, kCtasPerSm) void attn_block_kernel(KvView kv, BlockArgs a, unsigned* err) {
  constexpr int kStageBytes = 2 * kTile * D;
  constexpr int kPieces = D / 16;        // 16-byte pieces of a row
  constexpr int kRowsPer = 32 / kPieces; // rows one copy instruction of a warp covers
  constexpr int kChunks = D / 64;        // 64-channel parts of a row (4 pieces each)
  extern __shared__ __align__(1024) uint8_t ring[];
  __shared__ float s_ks[kWarps][kStages][kTile], s_vs[kWarps][kStages][kTile];
  __shared__ uint32_t s_live[kWarps][kStages];
  __shared__ float s_m[kWarps][8 * NT], s_l[kWarps][8 * NT];
  __shared__ Scan s_scan;
  __shared__ int s_last;
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c4 = lane & 3;
  const int G = kv.group, B = kv.block;
  const int pairs = kv.batch * kv.hkv, ctas = gridDim.x;

  int64_t per = 0, start = 0;
  int pair = 0;
  const int64_t total = sum_tiles(kv, a, s_scan, [&](int64_t all) {
    per = range_length(all, ctas);
    return static_cast<int64_t>(blockIdx.x) * per;
  }, &pair, &start);
  // pairs with nothing selected, and counts past the capacity
  for (int p = blockIdx.x; p < pairs; p += ctas) {
    const int raw = a.sel_count[p];
    if (raw > a.capacity && tid == 0) set_error(err, HS_EBIT_CAPACITY);
    if (raw > 0) continue;
    const int64_t b = p / kv.hkv, row = b * kv.hq + static_cast<int64_t>(p - b * kv.hkv) * G;
    for (int i = tid; i < G * D / 4; i += kThreads) store_out(a, row * D + 4 * i, make_float4(0.0f, 0.0f, 0.0f, 0.0f));
    if (a.lse && tid < G) a.lse[row + tid] = -INFINITY;
  }
  const int64_t t_begin = static_cast<int64_t>(blockIdx.x) * per;
  const int64_t t_end = min(total, t_begin + per);

  uint8_t* my_ring = ring + warp * (kStages * kStageBytes);
  const uint32_t my_ring_addr = smem_addr(my_ring);

  for (int64_t t = t_begin; t < t_end;) {
    // ---- the segment: tiles [seg0, seg1) of `pair` ----
    const int cnt = pair_count(kv, a, pair);
    const int64_t pair_tiles = tiles_of(kv, cnt);
    if (pair_tiles == 0) {
      ++pair;
      continue;
    }
    const int seg0 = static_cast<int>(t - start);
    const int seg1 = static_cast<int>(min(pair_tiles, t_end - start));
    const int b = pair / kv.hkv, kvh = pair - b * kv.hkv;
    const int L = kv.seq_lens[b];
    const int nb = min(ceil_div(max(L, 0), B), kv.max_blocks);
    const int32_t* sel = a.sel + static_cast<int64_t>(pair) * a.capacity;
    const int32_t* table = kv.page_table + static_cast<int64_t>(pair) * kv.max_blocks;

    // this lane's row of the warp's next tile to look up: selection entry, row in the block
    const int64_t u = static_cast<int64_t>(seg0 + warp) * kTile + lane;
    int ei = static_cast<int>(u / B), er = static_cast<int>(u - static_cast<int64_t>(ei) * B);
    const int step_i = kWarps * kTile / B, step_r = kWarps * kTile - step_i * B;
    const int tiles = seg0 + warp < seg1 ? (seg1 - seg0 - warp + kWarps - 1) / kWarps : 0;
    // lookups run ahead of the copies: the selected block one tile, its page another
    int left = tiles;               // tiles whose selection entry is still to be read
    int j1 = -1, r1 = 0;            // selected block (-1: none)
    int pg = -1, r2 = 0;            // page (-1: no row)
    auto look_sel = [&]() {
      j1 = -1;
      r1 = er;
      if (left > 0) {
        if (ei < cnt) {
          j1 = __ldg(sel + ei);
          if (j1 < 0 || j1 >= nb) {
            set_error(err, HS_EBIT_BLOCK_RANGE);
            j1 = -1;
          }
        }
        --left;
      }
      ei += step_i;
      er += step_r;
      if (er >= B) {
        er -= B;
        ++ei;
      }
    };
    auto look_page = [&]() {
      pg = -1;
      r2 = r1;
      if (j1 >= 0 && r1 < L - j1 * B) {
        pg = __ldg(table + j1);
        if (pg < 0 || pg >= kv.num_pages) {
          set_error(err, HS_EBIT_PAGE_RANGE);
          pg = -1;
        }
      }
    };
    int stage_in = 0;
    auto issue = [&]() {  // copies of the tile whose pages are known
      const uint32_t dst = my_ring_addr + stage_in * kStageBytes;
      const uint32_t live = __ballot_sync(0xffffffffu, pg >= 0);
      const int64_t row = pg >= 0 ? static_cast<int64_t>(pg) * B + r2 : 0;
#pragma unroll
      for (int i = 0; i < kTile / kRowsPer; ++i) {
        const int r = i * kRowsPer + lane / kPieces, c = lane % kPieces;
        const int64_t at = __shfl_sync(0xffffffffu, row, r) * D + 16 * c;
        const bool ok = (live >> r) & 1u;
        copy16(dst + piece_at<D>(r, c), static_cast<const uint8_t*>(kv.k_pages) + at, ok);
        copy16(dst + kTile * D + piece_at<D>(r, c), static_cast<const uint8_t*>(kv.v_pages) + at, ok);
      }
      const int pp = pg >= 0 ? pg : 0;
      copy4(smem_addr(&s_ks[warp][stage_in][lane]), kv.k_scales + pp, pg >= 0);
      copy4(smem_addr(&s_vs[warp][stage_in][lane]), kv.v_scales + pp, pg >= 0);
      if (lane == 0) s_live[warp][stage_in] = live;
      stage_in = stage_in + 1 == kStages ? 0 : stage_in + 1;
    };
    look_sel();
    look_page();
    look_sel();
    int issued = 0;
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
      if (issued < tiles) {
        issue();
        ++issued;
      }
      copies_commit();
      look_page();
      look_sel();
    }

    // ---- the query, as the S product's second operand ----
    uint32_t qf[NT][4 * kChunks][2];
    float qs[NT][2];  // logit factor of heads 2 c4, 2 c4 + 1 (log2 units)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int h = nt * 8 + g;
      float x[kChunks][16];
      float amax = 0.0f;
#pragma unroll
      for (int k = 0; k < kChunks; ++k) {
        if (h < G) {
          const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) +
                                                            (static_cast<int64_t>(b) * kv.hq + kvh * G + h) * D + 64 * k + 16 * c4);
          const uint4 v0 = __ldg(src), v1 = __ldg(src + 1);
          const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            x[k][2 * i] = __uint_as_float(w[i] << 16);
            x[k][2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            amax = fmaxf(amax, fmaxf(fabsf(x[k][2 * i]), fabsf(x[k][2 * i + 1])));
          }
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) x[k][i] = 0.0f;
        }
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      float f = 1.0f;  // 2^(7 - exponent of amax)
      if (amax > 0.0f && amax < INFINITY) f = __uint_as_float(static_cast<uint32_t>(min(254, 261 - static_cast<int>(__float_as_uint(amax) >> 23))) << 23);
#pragma unroll
      for (int k = 0; k < kChunks; ++k)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          qf[nt][4 * k + w][0] = pack_half2(x[k][4 * w] * f, x[k][4 * w + 1] * f);
          qf[nt][4 * k + w][1] = pack_half2(x[k][4 * w + 2] * f, x[k][4 * w + 3] * f);
        }
      const float s = a.scale * kLog2e / f;
      qs[nt][0] = __shfl_sync(0xffffffffu, s, 8 * c4);
      qs[nt][1] = __shfl_sync(0xffffffffu, s, 8 * c4 + 4);
    }

    float m[NT][2], l[NT][2];
    float o[NT][D / 16][4];
    float vref = kMinRef;  // power of two >= every V scale met
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.0f;
    }

    int stage = 0;
    for (int n = 0; n < tiles; ++n) {
      __syncwarp();  // the stage about to be filled has been read by every lane
      if (issued < tiles) {
        issue();
        ++issued;
      }
      copies_commit();
      look_page();
      look_sel();
      copies_wait<kStages - 1>();
      __syncwarp();
      const uint8_t* kt = my_ring + stage * kStageBytes;
      const uint8_t* vt = kt + kTile * D;
      const float* ks = s_ks[warp][stage];
      const float* vs = s_vs[warp][stage];
      const uint32_t live = s_live[warp][stage];

      // S = K Q^T
      float s[2][NT][4];
#pragma unroll
      for (int st = 0; st < 2; ++st) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[st][nt][e] = 0.0f;
        const int ra = 16 * st + token_of<D>(g), rb = ra + 8;
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
          const uint4 xa = *reinterpret_cast<const uint4*>(kt + piece_at<D>(ra, 4 * k + c4));
          const uint4 xb = *reinterpret_cast<const uint4*>(kt + piece_at<D>(rb, 4 * k + c4));
          const uint32_t wa[4] = {xa.x, xa.y, xa.z, xa.w}, wb[4] = {xb.x, xb.y, xb.z, xb.w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t a0 = lo2(wa[w]), a1 = lo2(wb[w]), a2 = hi2(wa[w]), a3 = hi2(wb[w]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma(s[st][nt], a0, a1, a2, a3, qf[nt][4 * k + w][0], qf[nt][4 * k + w][1]);
          }
        }
      }

      // logits (log2 units), their maximum over the tile
      float kr[4], vr[4];
      bool ok[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 8 * i + token_of<D>(g);
        kr[i] = ks[r];
        vr[i] = vs[r];
        ok[i] = (live >> r) & 1u;
      }
      bool raised = false;
      float mn[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float top = -INFINITY;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float& x = s[i >> 1][nt][2 * (i & 1) + e];
            x = ok[i] ? x * (kr[i] * qs[nt][e]) : -INFINITY;
            top = fmaxf(top, x);
          }
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
          mn[nt][e] = fmaxf(m[nt][e], top);
          raised |= mn[nt][e] > m[nt][e];
        }
      const uint32_t vmax = __reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(vs[lane])));
      const uint32_t vcap = max(__float_as_uint(vref), (vmax + 0x7fffffu) & 0x7f800000u);
      if (__any_sync(0xffffffffu, raised) || vcap != __float_as_uint(vref)) {
        const float vnew = __uint_as_float(vcap);
        const float down = vref / vnew;
        vref = vnew;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float f = m[nt][e] == -INFINITY ? 0.0f : exp2f(m[nt][e] - mn[nt][e]);
            l[nt][e] *= f;
            m[nt][e] = mn[nt][e];
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              o[nt][i][e] *= f * down;
              o[nt][i][2 + e] *= f * down;
            }
          }
      }
      const float unit = 16384.0f / vref;
#pragma unroll
      for (int i = 0; i < 4; ++i) vr[i] *= unit;

      // P, and O^T += V^T P^T
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float p[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float base = m[nt][e] == -INFINITY ? 0.0f : m[nt][e];
              p[e] = exp2f(s[st][nt][2 * i + e] - base);
              l[nt][e] += p[e];
              p[e] *= vr[2 * st + i];
            }
            const uint32_t hi = pack_half2(p[0], p[1]);
            const float2 back = unpack_half2(hi);
            ph[nt][i] = transpose8x8(hi);
            pl[nt][i] = transpose8x8(pack_half2(p[0] - back.x, p[1] - back.y));
          }
        const int t0 = 16 * st + token_of<D>(2 * c4), t1 = 16 * st + token_of<D>(2 * c4 + 1);
        constexpr int kWords = D / 32;  // words of a lane's channels: D / 8 of them
        uint32_t x[4][kWords];
        if constexpr (D == 128) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 v = *reinterpret_cast<const uint4*>(vt + piece_at<D>((i & 1 ? t1 : t0) + 8 * (i >> 1), g));
            x[i][0] = v.x; x[i][1] = v.y; x[i][2] = v.z; x[i][3] = v.w;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint2 v = *reinterpret_cast<const uint2*>(vt + piece_at<D>((i & 1 ? t1 : t0) + 8 * (i >> 1), g >> 1) + 8 * (g & 1));
            x[i][0] = v.x; x[i][1] = v.y;
          }
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const uint32_t pick = (i & 1) ? 0x7362u : 0x5140u;  // (byte of token 2k, byte of token 2k + 1) twice
          const uint32_t y0 = __byte_perm(x[0][i >> 1], x[1][i >> 1], pick), y1 = __byte_perm(x[2][i >> 1], x[3][i >> 1], pick);
          const uint32_t a0 = lo2(y0), a1 = hi2(y0), a2 = lo2(y1), a3 = hi2(y1);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma(o[nt][i], a0, a1, a2, a3, ph[nt][0], ph[nt][1]);
            mma(o[nt][i], a0, a1, a2, a3, pl[nt][0], pl[nt][1]);
          }
        }
      }
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    copies_wait<0>();

    // ---- the warps' states joined ----
    __syncthreads();  // every warp is done with its ring: it now holds the outputs
    float* so = reinterpret_cast<float*>(ring);  // [warp][8 NT][D]
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = l[nt][e];
        sum += __shfl_xor_sync(0xffffffffu, sum, 4);
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        const int h = nt * 8 + 2 * c4 + e;
        if (g == 0) {
          s_m[warp][h] = m[nt][e];
          s_l[warp][h] = sum;
        }
        const float back = vref * 6.103515625e-05f;  // 2^-14
        float* dst = so + (warp * 8 * NT + h) * D + g * (D / 8);
#pragma unroll
        for (int i = 0; i < D / 16; i += 2)
          *reinterpret_cast<float4*>(dst + 2 * i) =
              make_float4(o[nt][i][e] * back, o[nt][i][2 + e] * back, o[nt][i + 1][e] * back, o[nt][i + 1][2 + e] * back);
      }
    __syncthreads();
    const int c0 = static_cast<int>(start / per), c1 = static_cast<int>((start + pair_tiles - 1) / per);
    const bool whole = c0 == c1;
    const int64_t ws_row = (2 * static_cast<int64_t>(blockIdx.x) + (t_begin >= start ? 0 : 1)) * G;
    for (int idx = tid; idx < G * (D / 4); idx += kThreads) {
      const int h = idx / (D / 4), d = (idx - h * (D / 4)) * 4;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][h]);
      float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      float lse = -INFINITY;
      if (M != -INFINITY) {
        float tot = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float f = exp2f(s_m[w][h] - M);
          const float4 v = *reinterpret_cast<const float4*>(so + (w * 8 * NT + h) * D + d);
          tot = fmaf(s_l[w][h], f, tot);
          acc.x = fmaf(v.x, f, acc.x);
          acc.y = fmaf(v.y, f, acc.y);
          acc.z = fmaf(v.z, f, acc.z);
          acc.w = fmaf(v.w, f, acc.w);
        }
        acc = make_float4(acc.x / tot, acc.y / tot, acc.z / tot, acc.w / tot);
        lse = M * kLn2 + logf(tot);
      }
      if (whole) {
        const int64_t row = static_cast<int64_t>(b) * kv.hq + kvh * G + h;
        store_out(a, row * D + d, acc);
        if (d == 0 && a.lse) a.lse[row] = lse;
      } else {
        *reinterpret_cast<float4*>(a.ws_o + (ws_row + h) * D + d) = acc;
        if (d == 0) a.ws_lse[ws_row + h] = lse;
      }
    }
    if (!whole && a.counters) {
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        const uint32_t there = atomicAdd(a.counters + pair, 1u);
        s_last = there == static_cast<uint32_t>(c1 - c0);
        if (s_last) a.counters[pair] = 0u;
        __threadfence();
      }
      __syncthreads();
      if (s_last) merge_pair<D>(kv, a, pair, start, per, c0, c1);
    }
    __syncthreads();  // the ring and s_m are free again
    t = start + seg1;
    if (seg1 == pair_tiles) {
      start += pair_tiles;
      ++pair;
    }
  }
}

// The merge as a launch of its own, for callers without split counters.  CTA =
// pair.
template <int D>
__global__ __launch_bounds__(kThreads) void attn_block_merge_kernel(KvView kv, BlockArgs a, int ctas) {
  __shared__ Scan s_scan;
  pdl_trigger();
  pdl_wait();
  const int pair = blockIdx.x;
  const int64_t n = tiles_of(kv, pair_count(kv, a, pair));
  // the pair's first tile: the tiles of the pairs before it
  int64_t mine = 0;
  for (int p = threadIdx.x; p < kv.batch * kv.hkv; p += kThreads) {
    const int64_t k = tiles_of(kv, pair_count(kv, a, p));
    if (p < pair) mine += k;
  }
  mine = warp_sum(mine);
  if ((threadIdx.x & 31) == 0) s_scan.sums[threadIdx.x >> 5] = mine;
  __syncthreads();
  int64_t start = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) start += s_scan.sums[w];
  __syncthreads();
  int unused_pair;
  int64_t unused_start, per = 0;
  sum_tiles(kv, a, s_scan, [&](int64_t all) {
    per = range_length(all, ctas);
    return int64_t(0);
  }, &unused_pair, &unused_start);
  if (n == 0) return;
  const int c0 = static_cast<int>(start / per), c1 = static_cast<int>((start + n - 1) / per);
  if (c0 != c1) merge_pair<D>(kv, a, pair, start, per, c0, c1);
}

template <int D, int NT>
cudaError_t launch_n(const KvView& kv, const BlockArgs& b, int ctas, unsigned* err, cudaStream_t st) {
  auto kern = attn_block_kernel<D, NT>;
  if (cudaError_t e = allow_dynamic_smem(kern, ring_bytes<D>()); e != cudaSuccess) return e;
  cudaError_t e = launch_pdl(kern, dim3(ctas), dim3(kThreads), ring_bytes<D>(), st, kv, b, err);
  if (e != cudaSuccess || b.counters) return e;
  return launch_pdl(attn_block_merge_kernel<D>, dim3(kv.batch * kv.hkv), dim3(kThreads), 0, st, kv, b, ctas);
}

}  // namespace

int block_attn_ctas(int sms) { return sms * kCtasPerSm; }

cudaError_t launch_block_attn(const KvView& kv, const AttnArgs& a, unsigned* err, cudaStream_t st) {
  if (kv.batch == 0) return cudaSuccess;
  BlockArgs b;
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
  const int ctas = block_attn_ctas(a.sms);
  if (kv.head_dim == 128)
    return kv.group <= 8 ? launch_n<128, 1>(kv, b, ctas, err, st) : launch_n<128, 2>(kv, b, ctas, err, st);
  return kv.group <= 8 ? launch_n<64, 1>(kv, b, ctas, err, st) : launch_n<64, 2>(kv, b, ctas, err, st);
}

}  // namespace hs
