// Attention weights accumulated per token ("KV 稀疏化" wiki §2, H2O: the tokens that
// attention has looked at most are kept): for every token t of the selected blocks
//   weights[b][kvh][t] += sum over the group's heads of e^(scale q.K[t] - lse),
// lse being what the step's attention left, so that every head adds 1 in all.
//
// Every token's sum is formed once and by one lane, so nothing is normalised or merged:
// the 32-token tiles of all pairs' selections, end to end, are cut into one run for each
// warp.  A warp looks its rows up and copies them to its ring in shared memory as the
// attention over caches cut by counts does (attn_parts.cuh), K only.
//
// S[token][head] = K . Q^T on the warp-level matrix instruction m16n8k16: a token's
// heads lie in four lanes, which add their exponentials.  bf16 K and q as they are; e4m3
// codes as f16, and q times a power of two (exact within 2^-25 of the largest entry);
// 4-bit codes as bf16 numbers below the normal ones, as in the attention.  Scales of
// groups of channels are applied to the groups' partial sums.  f32 caches: on the CUDA
// cores, as fp32 products are wanted.
//
// What bounds it: memory for bf16 (16 requests x 4 heads x 16384 tokens, 277 MB: 46.3 us,
// 0.88 of the copy rate); instructions beside it for the others (4-bit, 32 requests, 185
// MB: 34.5 us, 0.79; e4m3 0.73 to 0.77); the CUDA cores for f32 (0.72).  A short call, 4
// requests of up to 3000 tokens, takes 4.3 us: the launch, the counts and one chain of
// lookups.
#include <limits.h>

#include "attn_parts.cuh"
#include "kv_row.cuh"

namespace hs {
namespace {

using namespace parts;

constexpr int kStages = 3;  // tiles in a warp's ring

template <int D, int KIND>
struct Row {
  static constexpr int kBytes = KIND == HS_KV_BF16 ? 2 * D : KIND == HS_KV_INT4_G32 ? D / 2 : D;
  static constexpr int kPieces = kBytes / 16;
  static constexpr bool kGrouped = KIND == HS_KV_FP8E4M3_G32 || KIND == HS_KV_INT4_G32;
  static constexpr int kRecord = kGrouped ? D / 8 : KIND == HS_KV_FP8E4M3_BLOCK ? 4 : 0;  // bytes of scales
  static constexpr int kStage = kTile * kBytes + (kRecord ? kTile * 16 : 0);
  // as many warps as the rings and 128 registers a thread allow
  static constexpr int kWarps = kBytes == 256 ? 8 : 16;
};

// Where 16-byte piece c of row r of a tile lies: 8 rows' piece c without bank conflicts.
template <int BYTES>
__device__ __forceinline__ uint32_t piece_at(int r, int c) {
  return r * BYTES + ((BYTES >= 128 ? c ^ (r & 7) : BYTES == 64 ? c ^ ((r >> 1) & 3) : c ^ ((r >> 2) & 1)) << 4);
}

// Selected blocks of a pair and their tiles.
__device__ __forceinline__ int blocks_of(const WeightsArgs& a, int64_t p) { return min(max(__ldg(a.sel_count + p), 0), a.capacity); }

// A warp's equal run of the tiles of all pairs, end to end.
struct TileRun {
  int pair, first, left;  // the pair, its first tile of the run, tiles of the run to come

  __device__ __forceinline__ TileRun(const KvView& kv, const WeightsArgs& a, int64_t w, int64_t warps, int lane) : pair(0), first(0), left(0) {
    const int pairs = kv.batch * kv.hkv, mine_n = (pairs + 31) / 32, p0 = min(pairs, lane * mine_n), p1 = min(pairs, p0 + mine_n);
    int64_t mine = 0;
    for (int p = p0; p < p1; ++p) mine += tiles_of(kv, blocks_of(a, p));
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const int64_t total = __shfl_sync(0xffffffffu, incl, 31), per = (total + warps - 1) / warps, g = w * per;
    if (g >= total) return;
    left = static_cast<int>(min(total - g, per));
    const int owner = __ffs(__ballot_sync(0xffffffffu, incl > g)) - 1;
    if (lane == owner) {
      int64_t before = incl - mine;
      for (pair = p0; pair < p1 - 1; ++pair) {
        const int n = tiles_of(kv, blocks_of(a, pair));
        if (g < before + n) break;
        before += n;
      }
      first = static_cast<int>(g - before);
    }
    pair = __shfl_sync(0xffffffffu, pair, owner);
    first = __shfl_sync(0xffffffffu, first, owner);
  }
  // Tiles of the run in this pair, then on to the next pair that has tiles.
  __device__ __forceinline__ int here(const KvView& kv, int count) const { return min(left, tiles_of(kv, count) - first); }
  __device__ __forceinline__ void on(const KvView& kv, const WeightsArgs& a, int n) {
    left -= n;
    first += n;
    while (left > 0 && first >= tiles_of(kv, blocks_of(a, pair))) {
      ++pair;
      first = 0;
    }
  }
};

__device__ __forceinline__ void report_counts(const KvView& kv, const WeightsArgs& a, unsigned* err) {
  if (blockIdx.x != 0) return;
  for (int p = threadIdx.x; p < kv.batch * kv.hkv; p += blockDim.x)
    if (__ldg(a.sel_count + p) > a.capacity) set_error(err, HS_EBIT_CAPACITY);
}

template <int D, int KIND, int NT>
__global__ __launch_bounds__(Row<D, KIND>::kWarps * 32, 1) void weights_kernel(KvView kv, WeightsArgs a, unsigned* err) {
  using R = Row<D, KIND>;
  constexpr int kWarps = R::kWarps, kBytes = R::kBytes, kRowsPer = 32 / R::kPieces;
  constexpr int kGroups = R::kGrouped ? D / kQuantGroup : 1;  // of channels with scales of their own
  constexpr int kSteps = D / 16, kEach = kSteps / kGroups;    // products over 16 channels
  extern __shared__ __align__(1024) uint8_t ring[];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c4 = lane & 3, mat = lane >> 3, mr = lane & 7;
  const int G = kv.group;
  report_counts(kv, a, err);
  uint8_t* my_ring = ring + warp * (kStages * R::kStage);
  const uint32_t ring_addr = smem_addr(my_ring);
  const uint8_t* piece = static_cast<const uint8_t*>(kv.k_pages) + 16 * (lane % R::kPieces);
  const uint8_t* records = reinterpret_cast<const uint8_t*>(kv.k_scales);
  const uint32_t my_at = piece_at<kBytes>(lane / R::kPieces, lane % R::kPieces);
  if constexpr (KIND == HS_KV_INT4_G32 && D == 64)  // the empty halves of the records
    for (int i = 0; i < kStages; ++i)
      *reinterpret_cast<uint2*>(my_ring + i * R::kStage + kTile * kBytes + lane * 16 + 8) = make_uint2(0u, 0u);

  TileRun run(kv, a, static_cast<int64_t>(warp) * gridDim.x + blockIdx.x, static_cast<int64_t>(gridDim.x) * kWarps, lane);
  while (run.left > 0) {
    const int cnt = blocks_of(a, run.pair);
    const int tiles = run.here(kv, cnt);
    const int b = run.pair / kv.hkv, kvh = run.pair - b * kv.hkv;
    TileRows<WeightsArgs> rows(kv, a, run.pair, cnt, __ldg(kv.seq_lens + b), run.first, tiles, lane, err);
    float* out = a.weights + static_cast<int64_t>(run.pair) * kv.max_blocks * kv.block;
    int stage_in = 0, place_in[kStages];
#pragma unroll
    for (int i = 0; i < kStages; ++i) place_in[i] = -1;
    // the copies of the next tile; the lane's token's place, -1 where there is none
    const auto issue = [&]() {
      uint32_t row;
      int place;
      const bool ok = rows.template next_at<true>(row, place);
      const uint32_t live = __ballot_sync(0xffffffffu, ok);
      const uint32_t dst = ring_addr + stage_in * R::kStage;
#pragma unroll
      for (int i = 0; i < kTile / kRowsPer; ++i) {
        const int r = i * kRowsPer + lane / R::kPieces;
        const uint64_t at = static_cast<uint64_t>(__shfl_sync(0xffffffffu, row, r)) * kBytes;
        // (rows are permuted by 8: pieces of 256-byte rows differ between copies)
        const uint32_t to = dst + (kRowsPer % 8 == 0 ? my_at + i * (kRowsPer * kBytes) : piece_at<kBytes>(r, lane % R::kPieces));
        copy16_if(to, piece + at, (live >> r) & 1u);
      }
      if constexpr (KIND == HS_KV_FP8E4M3_G32) {
        // one by one, as they may start at any element, and no slower (16 requests x 4 heads x
        // 16384 tokens 30.5 us, by 16 bytes 31.1; 32 x 8 x 32768 of 64 channels 108, by 8 bytes 111)
#pragma unroll
        for (int i = 0; i < R::kRecord; i += 4)
          copy4(dst + kTile * kBytes + lane * 16 + i, records + static_cast<uint64_t>(row) * R::kRecord + i, ok);
      } else if constexpr (R::kRecord == 16)
        copy16_if(dst + kTile * kBytes + lane * 16, records + static_cast<uint64_t>(row) * 16, ok);
      else if constexpr (R::kRecord == 8)
        copy8(dst + kTile * kBytes + lane * 16, records + static_cast<uint64_t>(row) * 8, ok);
      else if constexpr (R::kRecord == 4)
        copy4(dst + kTile * kBytes + lane * 16, records + static_cast<uint64_t>(row / static_cast<uint32_t>(kv.block)) * 4, ok);
      stage_in = stage_in + 1 == kStages ? 0 : stage_in + 1;
      return ok ? place : -1;
    };
    int issued = 0;
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
      if (issued < tiles) {
        place_in[i] = issue();
        ++issued;
      }
      copies_commit();
    }

    // ---- the query, as second operands, and what is added to a logit (log2 units) ----
    uint32_t qb[NT][kSteps][2];
    uint32_t xb[NT][3];        // 4-bit: what a record's scales and centres are multiplied by, as three bf16 terms
    float2 f[NT], minus[NT];   // heads 8 nt + 2 c4 and + 1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const bool head = nt * 8 + g < G;
      const int64_t at = static_cast<int64_t>(b) * kv.hq + kvh * G + nt * 8 + g;
      const uint16_t* src = static_cast<const uint16_t*>(a.q) + at * D;
      const float lse = head ? __ldg(a.lse + at) : -INFINITY;
      float factor = a.scale * kLog2e;
      if constexpr (KIND == HS_KV_BF16) {  // channels 16 i + 2 c4, + 1 and 8 more
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            qb[nt][i][h] = head ? __ldg(reinterpret_cast<const uint32_t*>(src + 16 * i + 8 * h + 2 * c4)) : 0u;
      } else if constexpr (KIND == HS_KV_INT4_G32) {  // channels 32 k + 8 c4 .. + 7
        uint4 raw[kGroups];
#pragma unroll
        for (int k = 0; k < kGroups; ++k)
          raw[k] = head ? __ldg(reinterpret_cast<const uint4*>(src + 32 * k + 8 * c4)) : make_uint4(0u, 0u, 0u, 0u);
        const Int4Query<kGroups> mine(raw, a.scale, c4);
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) qb[nt][i][h] = mine.q[i / 2][2 * (i % 2) + h];
#pragma unroll
        for (int i = 0; i < 3; ++i) xb[nt][i] = mine.terms[i];
        factor = mine.factor;
      } else {  // channels 16 i + 4 c4 .. + 3
        uint2 v[kSteps];
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          v[i] = head ? __ldg(reinterpret_cast<const uint2*>(src + 16 * i + 4 * c4)) : make_uint2(0u, 0u);
          amax = fmaxf(amax, fmaxf(fmaxf(fabsf(lower(v[i].x)), fabsf(upper(v[i].x))), fmaxf(fabsf(lower(v[i].y)), fabsf(upper(v[i].y)))));
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        float up = 1.0f;  // 2^(8 - exponent of amax), 2^127 at most
        if (amax > 0.0f && amax < INFINITY)
          up = __uint_as_float(static_cast<uint32_t>(min(254, 262 - static_cast<int>(__float_as_uint(amax) >> 23))) << 23);
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          qb[nt][i][0] = pack_half2(lower(v[i].x) * up, upper(v[i].x) * up);
          qb[nt][i][1] = pack_half2(lower(v[i].y) * up, upper(v[i].y) * up);
        }
        factor /= up;
      }
      // an empty head, or none: every weight of it is e^-inf
      const float less = lse == -INFINITY ? -INFINITY : -lse * kLog2e;
      f[nt] = make_float2(__shfl_sync(0xffffffffu, factor, 8 * c4), __shfl_sync(0xffffffffu, factor, 8 * c4 + 4));
      minus[nt] = make_float2(__shfl_sync(0xffffffffu, less, 8 * c4), __shfl_sync(0xffffffffu, less, 8 * c4 + 4));
    }

    int stage = 0;
    for (int n = 0; n < tiles; ++n) {
      __syncwarp();  // the stage about to be filled has been read by every lane
      const int place = place_in[0];
#pragma unroll
      for (int i = 0; i < kStages - 1; ++i) place_in[i] = place_in[i + 1];
      if (issued < tiles) {
        place_in[kStages - 2] = issue();
        ++issued;
      }
      copies_commit();
      copies_wait<kStages - 1>();
      __syncwarp();
      const uint32_t st = ring_addr + stage * R::kStage;
      const uint8_t* recs = my_ring + stage * R::kStage + kTile * kBytes;
      float sums[4];  // of tokens g, g + 8, g + 16, g + 24, this lane's heads
      uint32_t kr[4];
      if constexpr (KIND == HS_KV_INT4_G32) load4(st + kTile * kBytes + 16 * lane, kr);
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        float s[NT][kGroups][4], add[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            add[nt][e] = 0.0f;
#pragma unroll
            for (int k = 0; k < kGroups; ++k) s[nt][k][e] = 0.0f;
          }
        // a matrix of 8 rows and one piece to each 8 lanes: rows 0 and 8 on, the next piece of both
        const int r = 16 * mt + 8 * (mat & 1) + mr;
#pragma unroll
        for (int p = 0; p < R::kPieces; p += 2) {
          uint32_t w[4];
          load4(st + piece_at<kBytes>(r, p + (mat >> 1)), w);
          if constexpr (KIND == HS_KV_BF16) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_bf16(s[nt][0], w[0], w[1], w[2], w[3], qb[nt][p / 2][0], qb[nt][p / 2][1]);
          } else if constexpr (KIND == HS_KV_INT4_G32) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t x = w[2 * h], y = w[2 * h + 1], x8 = x >> 8, y8 = y >> 8;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma_bf16(s[nt][p + h], x & 0x000f000fu, y & 0x000f000fu, x8 & 0x000f000fu, y8 & 0x000f000fu, qb[nt][2 * (p + h)][0],
                         qb[nt][2 * (p + h)][1]);
                mma_bf16(s[nt][p + h], x & 0x00f000f0u, y & 0x00f000f0u, x8 & 0x00f000f0u, y8 & 0x00f000f0u, qb[nt][2 * (p + h) + 1][0],
                         qb[nt][2 * (p + h) + 1][1]);
              }
            }
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t a0, a1, a2, a3;
              e4m3x4_to_halves(w[2 * h], a0, a2);
              e4m3x4_to_halves(w[2 * h + 1], a1, a3);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma_f16(s[nt][(p + h) / kEach], a0, a1, a2, a3, qb[nt][p + h][0], qb[nt][p + h][1]);
            }
          }
        }
        if constexpr (KIND == HS_KV_INT4_G32) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_bf16(add[nt], kr[2 * mt], kr[2 * mt + 1], kr[2 * mt], kr[2 * mt + 1], xb[nt][0], xb[nt][1]);
            mma_bf16(add[nt], kr[2 * mt], kr[2 * mt + 1], 0u, 0u, xb[nt][2], 0u);
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {  // tokens g and g + 8
          const uint8_t* rec = recs + 16 * (16 * mt + 8 * e + g);
          float sc[4] = {1.0f, 1.0f, 1.0f, 1.0f};
          if constexpr (KIND == HS_KV_INT4_G32) {
            const uint2 two = *reinterpret_cast<const uint2*>(rec);
            sc[0] = lower(two.x);
            sc[1] = upper(two.x);
            sc[2] = lower(two.y);
            sc[3] = upper(two.y);
          } else if constexpr (KIND == HS_KV_FP8E4M3_G32) {
            if constexpr (D == 128) {
              const float4 four = *reinterpret_cast<const float4*>(rec);
              sc[0] = four.x;
              sc[1] = four.y;
              sc[2] = four.z;
              sc[3] = four.w;
            } else {
              const float2 two = *reinterpret_cast<const float2*>(rec);
              sc[0] = two.x;
              sc[1] = two.y;
            }
          } else if constexpr (KIND == HS_KV_FP8E4M3_BLOCK) {
            sc[0] = *reinterpret_cast<const float*>(rec);
          }
          float sum = 0.0f;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float2 x = make_float2(s[nt][0][2 * e], s[nt][0][2 * e + 1]);
            if constexpr (R::kRecord != 0) x = mul2(x, both(sc[0]));
#pragma unroll
            for (int k = 1; k < kGroups; ++k) x = fma2(make_float2(s[nt][k][2 * e], s[nt][k][2 * e + 1]), both(sc[k]), x);
            float2 plus = minus[nt];
            if constexpr (KIND == HS_KV_INT4_G32) plus = add2(plus, make_float2(add[nt][2 * e], add[nt][2 * e + 1]));
            x = fma2(x, f[nt], plus);
            // (of no head, or an empty one: 0 times an infinite K is not a number)
            sum += (minus[nt].x == -INFINITY ? 0.0f : exp2_fast(x.x)) + (minus[nt].y == -INFINITY ? 0.0f : exp2_fast(x.y));
          }
          sums[2 * mt + e] = sum;
        }
      }
      // added over the four lanes of a token; lane 4 g + c4 is left with token 8 c4 + g
      const bool odd = c4 & 1, high = c4 & 2;
      float u0 = odd ? sums[1] : sums[0], u1 = odd ? sums[3] : sums[2];
      u0 += __shfl_xor_sync(0xffffffffu, odd ? sums[0] : sums[1], 1);
      u1 += __shfl_xor_sync(0xffffffffu, odd ? sums[2] : sums[3], 1);
      float w = high ? u1 : u0;
      w += __shfl_xor_sync(0xffffffffu, high ? u0 : u1, 2);
      const int at = __shfl_sync(0xffffffffu, place, 8 * c4 + g);
      if (at >= 0) atomicAdd(out + at, w);  // (a block may be selected twice: equal sums, in either order)
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    copies_wait<0>();
    __syncwarp();
    run.on(kv, a, tiles);
  }
}

// f32: 8 lanes take a token, 4 D / 32 channels each, four tokens and four heads at a time.
// The lanes' parts of a logit are joined by halving the heads, so that two lanes form its
// exponential and not eight.  16 requests x 4 heads x 16384 tokens, 546 MB: 112 us, 0.72 of
// the copy rate (1 head 91, 16 heads 178, bound by the reads of the query and the
// shuffles).  (One head and two tokens at a time, every lane with the whole logit: 242; the
// query not in shared memory 122, and with 16 warps, which spill, 134; two tokens at a time
// 143; the next tile's rows prefetched into the L2 149.)
__host__ __device__ constexpr int warps_f32(int head_dim) { return head_dim == 128 ? 6 : 8; }  // two CTAs to an SM, without spilling
template <int D>
__global__ __launch_bounds__(warps_f32(D) * 32, 2) void weights_f32_kernel(KvView kv, WeightsArgs a, unsigned* err) {
  constexpr int C = D / 32;  // 16-byte pieces of a lane, 8 lanes apart
  constexpr int kTokens = 4, kHeads = 4, kWarps = warps_f32(D);
  __shared__ float4 s_q[kWarps][16 * D / 4];  // the pair's query
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane & 7;
  const bool upper = lane & 4, odd = lane & 2;
  const int my_head = (upper ? 2 : 0) + (odd ? 1 : 0);  // of four
  report_counts(kv, a, err);
  TileRun run(kv, a, static_cast<int64_t>(warp) * gridDim.x + blockIdx.x, static_cast<int64_t>(gridDim.x) * kWarps, lane);
  while (run.left > 0) {
    const int cnt = blocks_of(a, run.pair), tiles = run.here(kv, cnt);
    const int b = run.pair / kv.hkv, kvh = run.pair - b * kv.hkv, G = kv.group;
    TileRows<WeightsArgs> rows(kv, a, run.pair, cnt, __ldg(kv.seq_lens + b), run.first, tiles, lane, err);
    float* out = a.weights + static_cast<int64_t>(run.pair) * kv.max_blocks * kv.block;
    const int64_t head0 = static_cast<int64_t>(b) * kv.hq + kvh * G;
    __syncwarp();
    for (int i = lane; i < G * (D / 4); i += 32) s_q[warp][i] = __ldg(reinterpret_cast<const float4*>(a.q) + head0 * (D / 4) + i);
    __syncwarp();
    const float4* q0 = s_q[warp] + c;
    for (int n = 0; n < tiles; ++n) {
      uint32_t row;
      int place;
      const bool ok = rows.template next_at<true>(row, place);
      if (__ballot_sync(0xffffffffu, ok) == 0u) continue;  // (there is a row 0 else, read where a token is not there)
      float sum = 0.0f;                                    // of token `lane`
#pragma unroll 1
      for (int t0 = 0; t0 < kTile; t0 += 4 * kTokens) {
        float4 x[kTokens][C];  // of token t0 + 4 t + lane / 8
#pragma unroll
        for (int t = 0; t < kTokens; ++t) {
          const uint32_t r = __shfl_sync(0xffffffffu, row, t0 + 4 * t + (lane >> 3));
          const float4* src = reinterpret_cast<const float4*>(kv.k_pages) + static_cast<uint64_t>(r) * (D / 4) + c;
#pragma unroll
          for (int k = 0; k < C; ++k) x[t][k] = __ldg(src + 8 * k);
        }
        float all[kTokens] = {};
#pragma unroll 1
        for (int h0 = 0; h0 < G; h0 += kHeads) {
          float dot[kHeads][kTokens];
#pragma unroll
          for (int h = 0; h < kHeads; ++h) {
            const float4* q = q0 + min(h0 + h, G - 1) * (D / 4);
            float2 two[kTokens];
#pragma unroll
            for (int t = 0; t < kTokens; ++t) two[t] = both(0.0f);
#pragma unroll
            for (int k = 0; k < C; ++k) {
              const float4 y = q[8 * k];
#pragma unroll
              for (int t = 0; t < kTokens; ++t) {
                two[t] = fma2(make_float2(x[t][k].x, x[t][k].y), make_float2(y.x, y.y), two[t]);
                two[t] = fma2(make_float2(x[t][k].z, x[t][k].w), make_float2(y.z, y.w), two[t]);
              }
            }
#pragma unroll
            for (int t = 0; t < kTokens; ++t) dot[h][t] = two[t].x + two[t].y;
          }
          const float lse = h0 + my_head < G ? __ldg(a.lse + head0 + h0 + my_head) : -INFINITY;
#pragma unroll
          for (int t = 0; t < kTokens; ++t) {
            float u = upper ? dot[2][t] : dot[0][t], v = upper ? dot[3][t] : dot[1][t];
            u += __shfl_xor_sync(0xffffffffu, upper ? dot[0][t] : dot[2][t], 4);
            v += __shfl_xor_sync(0xffffffffu, upper ? dot[1][t] : dot[3][t], 4);
            float z = odd ? v : u;
            z += __shfl_xor_sync(0xffffffffu, odd ? u : v, 2);
            z += __shfl_xor_sync(0xffffffffu, z, 1);
            if (lse != -INFINITY) all[t] += expf(fmaf(z, a.scale, -lse));
          }
        }
#pragma unroll
        for (int t = 0; t < kTokens; ++t) {
          all[t] += __shfl_xor_sync(0xffffffffu, all[t], 2);
          all[t] += __shfl_xor_sync(0xffffffffu, all[t], 4);
          const float v = __shfl_sync(0xffffffffu, all[t], 8 * (lane & 3));
          if (lane >> 2 == t0 / 4 + t) sum = v;
        }
      }
      if (ok) atomicAdd(out + place, sum);
    }
    run.on(kv, a, tiles);
  }
}

template <int D, int KIND, int NT>
cudaError_t launch_n(const KvView& kv, const WeightsArgs& a, int sms, unsigned* err, cudaStream_t st) {
  using R = Row<D, KIND>;
  constexpr size_t smem = static_cast<size_t>(R::kWarps) * kStages * R::kStage;
  auto kern = weights_kernel<D, KIND, NT>;
  static std::atomic<uint64_t> allowed{0};
  if (cudaError_t e = allow_dynamic_smem_once(allowed, kern, smem); e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(sms), dim3(R::kWarps * 32), smem, st, kv, a, err);
}

template <int D, int KIND>
cudaError_t launch_k(const KvView& kv, const WeightsArgs& a, int sms, unsigned* err, cudaStream_t st) {
  return kv.group <= 8 ? launch_n<D, KIND, 1>(kv, a, sms, err, st) : launch_n<D, KIND, 2>(kv, a, sms, err, st);
}

template <int D>
cudaError_t launch_d(const KvView& kv, const WeightsArgs& a, int sms, unsigned* err, cudaStream_t st) {
  switch (kv.kv_dtype) {
    case HS_KV_F32: return launch_pdl(weights_f32_kernel<D>, dim3(2 * sms), dim3(warps_f32(D) * 32), 0, st, kv, a, err);
    case HS_KV_BF16: return launch_k<D, HS_KV_BF16>(kv, a, sms, err, st);
    case HS_KV_FP8E4M3_G32: return launch_k<D, HS_KV_FP8E4M3_G32>(kv, a, sms, err, st);
    case HS_KV_INT4_G32: return launch_k<D, HS_KV_INT4_G32>(kv, a, sms, err, st);
    default: return launch_k<D, HS_KV_FP8E4M3_BLOCK>(kv, a, sms, err, st);
  }
}

}  // namespace

bool weights_fits(const KvView& kv, const WeightsArgs& a) {
  const int64_t pairs = static_cast<int64_t>(kv.batch) * kv.hkv, tokens = static_cast<int64_t>(a.capacity) * kv.block;
  return pairs <= INT32_MAX && kv.num_pages * kv.block <= UINT32_MAX && tokens <= INT32_MAX &&  // rows and places are 32-bit
         static_cast<int64_t>(kv.max_blocks) * kv.block <= INT32_MAX &&
         (tokens / kTile + 1) * pairs <= INT32_MAX;  // tiles
}

cudaError_t launch_weights(const KvView& kv, const WeightsArgs& a, int sms, unsigned* err, cudaStream_t st) {
  if (kv.batch == 0) return cudaSuccess;
  return kv.head_dim == 128 ? launch_d<128>(kv, a, sms, err, st) : launch_d<64>(kv, a, sms, err, st);
}

}  // namespace hs
