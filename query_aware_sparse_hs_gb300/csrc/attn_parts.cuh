// What the attention kernels that cut their work by the actual counts share: the parts
// of every (request, kv head)'s selection and the teams of warps that take them, the
// lookup of a run's rows, the merge of a pair's partial results.  Everything is in an
// anonymous namespace of its includer.
#pragma once

#include <limits.h>

#include "hs_internal.h"

namespace hs {
namespace {
namespace parts {

constexpr int kTeamWarps = 4;
constexpr int kMaxWarps = 4 * kTeamWarps;
constexpr int kTile = 32;       // tokens a warp handles at a time
constexpr int kMinTiles = 8;    // tiles of a part of a cut pair at least
// Pairs of up to so many tiles are not cut: two for each warp of a CTA (4 pairs of
// 1000 tokens, 128 channels, 32 tiles: 9.6 us cut, 11.0 whole; 16 tiles: 8.4 whole).
__host__ __device__ constexpr int whole_tiles(int teams) { return 2 * teams * kTeamWarps; }
constexpr int kMergeTiles = 3;  // what a merge costs, in tiles per warp
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMinRef = 1.925929944387236e-34f;  // 2^-112
constexpr uint32_t kMaxRef = 0x7f000000u;          // 2^127, as bits
// P * vscale enters in units of 2^-kUnit times the reference: 2^14 at most, twice that
// for a V scale above 2^127, which f16 holds.  (P up to 2^6, in units of 2^-8, would
// spare most rescalings of the state, 2% for 16 heads of 64 channels, for 6 bits less
// below the f16 range.)
constexpr int kUnit = 14;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// 16 bytes to shared memory
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// the same; zeros, and nothing read, unless `live`
__device__ __forceinline__ void copy16_if(uint32_t dst, const void* src, bool live) {
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
__device__ __forceinline__ float exp2_fast(float x) {  // 2 ulp; results under 2^-126 are 0
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 2^kUnit / ref, of a power of two from kMinRef to 2^127
__device__ __forceinline__ float unit_over(float ref) {
  return __uint_as_float((static_cast<uint32_t>(254 + kUnit) << 23) - __float_as_uint(ref));
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_half2(uint32_t w) { return __half22float2(*reinterpret_cast<__half2*>(&w)); }

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
// d = a b
__device__ __forceinline__ void mma_bf16_0(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
// d += a b
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
// x less two bf16, less two f16, without widening them first (16 heads of 64 channels 135 us
// for 139, of 128 channels 254 for 255; 8 heads of 64 channels 209 for 206)
__device__ __forceinline__ float2 less_bf16(float2 x, uint32_t two) {
  float2 d;
  asm("{\n\t.reg .b16 a, b, m;\n\tmov.b32 {a, b}, %2;\n\tmov.b16 m, 0xbf80;\n\tfma.rn.f32.bf16 %0, a, m, %3;\n\tfma.rn.f32.bf16 %1, b, m, %4;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "r"(two), "f"(x.x), "f"(x.y));
  return d;
}
__device__ __forceinline__ float2 less_f16(float2 x, uint32_t two) {
  float2 d;
  asm("{\n\t.reg .b16 a, b, m;\n\tmov.b32 {a, b}, %2;\n\tmov.b16 m, 0xbc00;\n\tfma.rn.f32.f16 %0, a, m, %3;\n\tfma.rn.f32.f16 %1, b, m, %4;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "r"(two), "f"(x.x), "f"(x.y));
  return d;
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
// Two fp32 numbers at a time.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\tfma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// A head's query for products with 4-bit codes, 8 channels (32 k + 8 c4 .. + 7) of every
// group k to a lane, the head's four lanes together.
template <int GROUPS>
struct Int4Query {
  uint32_t q[GROUPS][4];  // bf16 times 2^e: channels 0 4, 2 6 of the 8; by 1/16, as their codes are 16 times as large, 1 5, 3 7
  uint32_t terms[3];      // what word c4 of a record is multiplied by, in three bf16 terms: -8 sum q for a scale, sum q for a centre
  float factor;           // from the products with codes n 2^-133 to a logit (log2 units)

  __device__ __forceinline__ Int4Query(const uint4 (&raw)[GROUPS], float scale, int c4) {
    float amax = 0.0f, sum[GROUPS], x[GROUPS][8];
#pragma unroll
    for (int k = 0; k < GROUPS; ++k) {
      const uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
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
    // the largest entry in [2^100, 2^101) where e is from 10 to 127
    const int e = min(max(227 - static_cast<int>(__float_as_uint(amax) >> 23), 10), 127);
    const float up = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
    factor = scale * kLog2e * __uint_as_float(static_cast<uint32_t>(133 - e + 127) << 23);
#pragma unroll
    for (int k = 0; k < GROUPS; ++k) {
      q[k][0] = pack_bf16(x[k][0] * up, x[k][4] * up);
      q[k][1] = pack_bf16(x[k][2] * up, x[k][6] * up);
      q[k][2] = pack_bf16(x[k][1] * up * 0.0625f, x[k][5] * up * 0.0625f);
      q[k][3] = pack_bf16(x[k][3] * up * 0.0625f, x[k][7] * up * 0.0625f);
    }
    constexpr int kWords = GROUPS / 2;  // a record's words of scales; then those of centres
    const int pair = c4 & (kWords - 1);
    const float by = scale * kLog2e * (c4 < kWords ? -8.0f : c4 < 2 * kWords ? 1.0f : 0.0f);
    float r0 = (pair ? sum[GROUPS - 2] : sum[0]) * by, r1 = (pair ? sum[GROUPS - 1] : sum[1]) * by;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      terms[i] = pack_bf16(r0, r1);
      r0 -= lower(terms[i]);
      r1 -= upper(terms[i]);
    }
  }
};

struct PartArgs {
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

// Selected blocks of pair p, and tiles of so many.
__device__ __forceinline__ int pair_count(const PartArgs& a, int64_t p) {
  const int c = __ldg(a.sel_count + p);
  return min(max(c, 0), a.capacity);
}
__device__ __forceinline__ int tiles_of(const KvView& kv, int count) {  // (the host saw that all of them fit)
  return static_cast<int>((static_cast<uint32_t>(count) * kv.block + kTile - 1) / kTile);
}

// Warps that take parts together.  bar: 0 for the whole CTA, else the number of
// the hardware barrier.
struct Team {
  int rank, warps, bar;  // the thread's number in the team, the team's warps
  __device__ __forceinline__ int threads() const { return warps * 32; }
  __device__ __forceinline__ void sync() const {
    if (bar == 0)
      __syncthreads();
    else
      asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(kTeamWarps * 32) : "memory");
  }
};

// Every pair is cut into equal parts of at most `per` tiles; the parts of all
// pairs are numbered through and dealt to the slots in turn.  A slot is a team
// of kTeamWarps warps, or (joint) all warps of a CTA.  With
// per = total / max(slots - pairs, slots / 2) there are no more parts than slots
// where the pairs leave room for that (sum of ceil(n / per) <= total / per +
// pairs), and a long pair among many short ones is still spread over half the
// slots.  Short pairs are not cut: they have nothing to merge.  A pair that is cut
// has a row of the workspace for each part: at most 2 total / per <= 2 slots rows
// in all.
//   Joint parts halve (64 channels: third) the parts, and so the merges, and the
//   time of a short part; with more pairs than CTAs, or pairs so uneven that CTAs
//   are left idle, teams balance better.  Taken where every CTA has one part at
//   most and the longest pair's, in tiles per warp, is not longer than the teams' by
//   more than a merge.  With one term of P, 32 requests x 4 heads x 4096 selected tokens:
//   joint 28 us, teams 32; 24 uneven requests x 4 heads: 56 and 48; 64 x 4 heads x 4096:
//   54 and 49.
struct Cut {
  int per, slots, whole;
  bool joint;
};
struct Part {
  int pair;
  int index, count;  // which of the pair's parts
  int row;           // workspace row of the pair's first part
};
struct Pairs {  // one pair's numbers
  int part, count, row;  // its first part, how many, workspace row of the first
};
constexpr int kListed = 32;  // parts a team notes at a time

__device__ __forceinline__ int parts_of(int tiles, int per, int whole) {
  return tiles <= whole ? (tiles > 0 ? 1 : 0) : (tiles + per - 1) / per;
}
__device__ __forceinline__ int part_of(int tiles, int per) {  // the longest part of a pair that is cut
  const int k = max((tiles + per - 1) / per, 1);
  return (tiles + k - 1) / k;
}
__device__ __forceinline__ int per_of(int total, int pairs, int slots) {
  return max((total - 1) / max(max(slots - pairs, slots / 2), 1) + 1, kMinTiles);
}

struct Scratch {
  int64_t sums[kMaxWarps];
  int tiles[kMaxWarps], longest[kMaxWarps];
};

// The cut for this call's counts, by all threads of a CTA (`cta`).  seen(p, count)
// sees every pair once, in one of the threads.
template <typename F>
__device__ Cut choose_cut(const KvView& kv, const PartArgs& a, int ctas, int teams, const Team& cta, Scratch& sc, F&& seen) {
  const int warp = cta.rank >> 5, lane = cta.rank & 31;
  const int pairs = kv.batch * kv.hkv, mine_n = (pairs + cta.threads() - 1) / cta.threads();
  const int p0 = min(pairs, cta.rank * mine_n), p1 = min(pairs, p0 + mine_n);
  int total = 0, longest = 0;  // tiles
  for (int p = p0; p < p1; ++p) {
    const int c = pair_count(a, p), n = tiles_of(kv, c);
    seen(p, c);
    total += n;
    longest = max(longest, n);
  }
  total = __reduce_add_sync(0xffffffffu, total);
  longest = __reduce_max_sync(0xffffffffu, longest);
  if (lane == 0) {
    sc.tiles[warp] = total;
    sc.longest[warp] = longest;
  }
  cta.sync();
  total = longest = 0;
  for (int w = 0; w < cta.warps; ++w) {
    total += sc.tiles[w];
    longest = max(longest, sc.longest[w]);
  }
  const int per_joint = per_of(total, pairs, ctas), per_team = per_of(total, pairs, ctas * teams);
  Cut cut;
  cut.whole = whole_tiles(teams);
  // no more joint parts than CTAs: the pairs leave room for the cuts, or none is cut
  const bool one_each = pairs <= ctas / 2 || (pairs <= ctas && longest <= max(per_joint, cut.whole));
  const int joint = part_of(longest, per_joint), team = part_of(longest, per_team);
  cut.joint = one_each && joint <= (team / kTeamWarps + kMergeTiles) * kTeamWarps * teams;
  cut.slots = cut.joint ? ctas : ctas * teams;
  cut.per = cut.joint ? per_joint : per_team;
  return cut;
}

// each(p, numbers) sees every pair once, in one of the team's threads; the team
// meets before the number of parts is returned.
template <typename F>
__device__ int number_parts(const KvView& kv, const PartArgs& a, const Cut& cut, const Team& team, Scratch& sc, F&& each) {
  const int warp = team.rank >> 5, lane = team.rank & 31;
  const int pairs = kv.batch * kv.hkv, mine_n = (pairs + team.threads() - 1) / team.threads();
  const int p0 = min(pairs, team.rank * mine_n), p1 = min(pairs, p0 + mine_n);
  int64_t mine = 0;  // parts, and rows of the workspace in the upper half
  int k = 0;
  for (int p = p0; p < p1; ++p) {
    k = parts_of(tiles_of(kv, pair_count(a, p)), cut.per, cut.whole);
    mine += k + (k > 1 ? static_cast<int64_t>(k) << 32 : 0);
  }
  int64_t at = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, at, o);
    if (lane >= o) at += v;
  }
  if (lane == 31) sc.sums[warp] = at;
  at -= mine;
  team.sync();
  int64_t all = 0;
  for (int w = 0; w < team.warps; ++w) {
    if (w == warp) at += all;
    all += sc.sums[w];
  }
  for (int p = p0; p < p1; ++p) {
    Pairs n;
    n.count = mine_n == 1 ? k : parts_of(tiles_of(kv, pair_count(a, p)), cut.per, cut.whole);
    n.part = static_cast<int>(at & 0xffffffff);
    n.row = static_cast<int>(at >> 32);
    each(p, n);
    at += n.count + (n.count > 1 ? static_cast<int64_t>(n.count) << 32 : 0);
  }
  team.sync();
  return static_cast<int>(all & 0xffffffff);
}

__device__ __forceinline__ void store_out(const PartArgs& a, int64_t at, float4 v) {
  if (a.out_f32) {
    reinterpret_cast<float4*>(a.out)[at / 4] = v;
  } else {
    const __nv_bfloat162 x = __floats2bfloat162_rn(v.x, v.y), y = __floats2bfloat162_rn(v.z, v.w);
    reinterpret_cast<uint2*>(a.out)[at / 4] =
        make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
  }
}

// Joins the partial results of a pair into out / lse, every kTeamWarps warps of
// the team those of every groups-th part, and then the groups.  The order goes by
// the parts' numbers alone.  w: shared memory for G * (count + 1) floats and
// groups - 1 results.  The first results are on their way while their weights are
// found.
template <int D, int NT>
__device__ void merge_pair(const KvView& kv, const PartArgs& a, const Team& team, int64_t pair, int row0, int count,
                           float* w) {
  constexpr int kGroup = kTeamWarps * 32;
  constexpr int NI = NT * 8 * D / 4 / kGroup;  // 16-byte pieces of a result per thread, at most
  constexpr int U = 16 / NI;                   // results in flight
  const int G = kv.group, lane = team.rank & 31, warp = team.rank >> 5, threads = team.threads();
  const int groups = team.warps / kTeamWarps, grp = team.rank / kGroup, rank = team.rank - grp * kGroup;
  float* lses = w + G * count;
  float4* sums = reinterpret_cast<float4*>(w + (G * (count + 1) + 3) / 4 * 4);
  const float* ws_lse = a.ws_lse + static_cast<int64_t>(row0) * G;
  const float4* ws_o = reinterpret_cast<const float4*>(a.ws_o + static_cast<int64_t>(row0) * G * D);
  const int pieces = G * (D / 4);
  float4 got[U][NI];
  const auto load = [&](int i0) {
#pragma unroll
    for (int k = 0; k < U; ++k)
#pragma unroll
      for (int n = 0; n < NI; ++n) {
        const int i = i0 + k * groups, idx = rank + n * kGroup;
        got[k][n] = i < count && idx < pieces ? __ldcg(ws_o + static_cast<int64_t>(i) * pieces + idx)
                                              : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      }
  };
  load(grp);
  for (int i = team.rank; i < G * count; i += threads) w[i] = __ldcg(ws_lse + i);
  team.sync();
  for (int h = warp; h < G; h += team.warps) {
    float M = -INFINITY, tot = 0.0f;
    for (int i = lane; i < count; i += 32) M = fmaxf(M, w[i * G + h]);
    M = warp_max(M);
    if (M == -INFINITY) M = 0.0f;  // no token, or only results that are not numbers: those stay so
    for (int i = lane; i < count; i += 32) {
      const float e = expf(w[i * G + h] - M);
      w[i * G + h] = e;
      tot += e;
    }
    tot = warp_sum(tot);
    const float norm = tot == 0.0f ? 0.0f : 1.0f / tot;
    for (int i = lane; i < count; i += 32) w[i * G + h] *= norm;
    if (lane == 0) lses[h] = tot == 0.0f ? -INFINITY : M + logf(tot);
  }
  team.sync();
  float4 acc[NI];
#pragma unroll
  for (int n = 0; n < NI; ++n) acc[n] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int i0 = grp; i0 < count;) {
#pragma unroll
    for (int k = 0; k < U; ++k)
#pragma unroll
      for (int n = 0; n < NI; ++n) {
        const int i = i0 + k * groups, idx = rank + n * kGroup;
        const float e = i < count && idx < pieces ? w[i * G + idx / (D / 4)] : 0.0f;
        acc[n].x = fmaf(e, got[k][n].x, acc[n].x);
        acc[n].y = fmaf(e, got[k][n].y, acc[n].y);
        acc[n].z = fmaf(e, got[k][n].z, acc[n].z);
        acc[n].w = fmaf(e, got[k][n].w, acc[n].w);
      }
    i0 += U * groups;
    if (i0 < count) load(i0);
  }
  if (groups > 1) {
#pragma unroll
    for (int n = 0; n < NI; ++n)
      if (grp > 0 && rank + n * kGroup < pieces) sums[(grp - 1) * pieces + rank + n * kGroup] = acc[n];
    team.sync();
  }
  const int64_t b = pair / kv.hkv, out_row = b * kv.hq + (pair - b * kv.hkv) * G;
#pragma unroll
  for (int n = 0; n < NI; ++n) {
    const int idx = rank + n * kGroup;
    if (grp > 0 || idx >= pieces) continue;
    for (int j = 0; j < groups - 1; ++j) {
      const float4 v = sums[j * pieces + idx];
      acc[n] = make_float4(acc[n].x + v.x, acc[n].y + v.y, acc[n].z + v.z, acc[n].w + v.w);
    }
    store_out(a, out_row * D + 4 * idx, acc[n]);
  }
  if (a.lse && team.rank < G) a.lse[out_row + team.rank] = lses[team.rank];
}

// Pairs that nothing is selected of: out = 0, lse = -inf.  CTAs share them.
template <int D>
__device__ void answer_empty(const KvView& kv, const PartArgs& a, int tid, int threads) {
  const int G = kv.group;
  for (int p = blockIdx.x; p < kv.batch * kv.hkv; p += gridDim.x) {
    if (pair_count(a, p) > 0) continue;
    const int64_t b = p / kv.hkv, row = b * kv.hq + static_cast<int64_t>(p - b * kv.hkv) * G;
    for (int i = tid; i < G * D / 4; i += threads) store_out(a, row * D + 4 * i, make_float4(0.0f, 0.0f, 0.0f, 0.0f));
    if (a.lse && tid < G) a.lse[row + tid] = -INFINITY;
  }
}

// The states of a team's warps joined: running maxima, sums and references in s_m, s_l
// and s_ref by the team's warps, outputs in `so` ([warp][8 NT][D], in units of
// 2^-kUnit of the warp's reference).  A part that is a whole pair goes to out / lse,
// another to its row of the workspace, and the team that arrives last merges the pair.
template <int D, int NT>
__device__ void finish_part(const KvView& kv, const PartArgs& a, const Team& team, const Part& part, const float (*s_m)[8 * NT],
                            const float (*s_l)[8 * NT], const float* s_ref, float* so, int* last) {
  const int G = kv.group, b = part.pair / kv.hkv, ws_row = (part.row + part.index) * G;
  const bool whole = part.count == 1;
  for (int idx = team.rank; idx < G * (D / 4); idx += team.threads()) {
    const int h = idx / (D / 4), d = (idx - h * (D / 4)) * 4;
    float M = -INFINITY, ref = kMinRef;
    for (int w = 0; w < team.warps; ++w) {
      M = fmaxf(M, s_m[w][h]);
      ref = fmaxf(ref, s_ref[w]);
    }
    if (M == -INFINITY) M = 0.0f;  // no token, or only logits that are not numbers
    const float per = unit_over(ref);
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float tot = 0.0f;
#pragma unroll 4
    for (int w = 0; w < team.warps; ++w) {
      const float f = exp2f(s_m[w][h] - M);
      const float4 v = *reinterpret_cast<const float4*>(so + (w * 8 * NT + h) * D + d);
      const float fr = f * (s_ref[w] * per);  // (the sums stay in units of the largest reference)
      tot = fmaf(s_l[w][h], f, tot);
      acc.x = fmaf(v.x, fr, acc.x);
      acc.y = fmaf(v.y, fr, acc.y);
      acc.z = fmaf(v.z, fr, acc.z);
      acc.w = fmaf(v.w, fr, acc.w);
    }
    float lse = -INFINITY;
    if (tot != 0.0f) {
      const float n = 1.0f / (1 << 2 * kUnit) / tot;
      acc = make_float4(acc.x * n * ref, acc.y * n * ref, acc.z * n * ref, acc.w * n * ref);
      lse = M * kLn2 + logf(tot);
    }
    if (whole) {
      const int64_t row = static_cast<int64_t>(b) * kv.hq + (part.pair - b * kv.hkv) * G + h;
      store_out(a, row * D + d, acc);
      if (d == 0 && a.lse) a.lse[row] = lse;
    } else {
      *reinterpret_cast<float4*>(a.ws_o + static_cast<int64_t>(ws_row + h) * D + d) = acc;
      if (d == 0) a.ws_lse[ws_row + h] = lse;
    }
  }
  if (!whole && a.counters) {
    team.sync();
    if (team.rank == 0) {
      // releases what the team wrote before the barrier, acquires what the others released
      uint32_t there;
      asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(there) : "l"(a.counters + part.pair) : "memory");
      *last = there == static_cast<uint32_t>(part.count - 1);
      if (*last) a.counters[part.pair] = 0u;
    }
    team.sync();
    if (*last) merge_pair<D, NT>(kv, a, team, part.pair, part.row, part.count, so);
  }
}

// The merge as a launch of its own, for callers without split counters.  CTA =
// pair; as many warps as merge in place, so that the results are the same.
template <int D, int NT, int TEAMS>
__global__ __launch_bounds__(TEAMS * kTeamWarps * 32) void merge_parts_kernel(KvView kv, PartArgs a, int ctas) {
  extern __shared__ __align__(16) float weights[];
  __shared__ Scratch s_scratch;
  __shared__ Pairs s_pair;
  pdl_trigger();
  pdl_wait();
  const int pair = blockIdx.x, tid = threadIdx.x;
  const Team cta{tid, TEAMS * kTeamWarps, 0};
  const Cut cut = choose_cut(kv, a, ctas, TEAMS, cta, s_scratch, [](int, int) {});
  if (!cut.joint && tid >= kTeamWarps * 32) return;
  const Team team = cut.joint ? cta : Team{tid, kTeamWarps, 1};
  number_parts(kv, a, cut, team, s_scratch, [&](int p, const Pairs& n) {
    if (p == pair) s_pair = n;
  });
  if (s_pair.count > 1) merge_pair<D, NT>(kv, a, team, pair, s_pair.row, s_pair.count, weights);
}

// The rows of a run of 32-token tiles of a pair's selection, lane = token: which row of
// the pool it is, tile by tile.  Selected blocks are looked up 32 at a time, one to a
// lane, the pages one window ahead of the rows and the selection two, so that neither
// load is waited for.  A window holds the entries from that of its first tile on; a
// tile that does not fit opens the next.  All 32 lanes call everything.
// `Args` has sel and capacity.  (What a window that opens needs, and little else does, is
// worked out again then: registers are short where this is used.)
template <typename Args>
struct TileRows {
  const KvView& kv;
  const Args& a;
  unsigned* err;
  int64_t pair;
  uint32_t u, u_stop, w_end, e_base;  // the next tile's first token, the run's end, the window's end and first entry
  int lane, cnt, L, page, lim, page1, lim1, j0, j1, j2, ei, er, step_i, step_r;

  __device__ __forceinline__ uint32_t window_end(uint32_t from, uint32_t e) const {  // past the window's whole tiles
    return from + ((e + 32) * kv.block - from) / kTile * kTile;
  }
  __device__ __forceinline__ int load_sel(uint32_t from, uint32_t e) const {  // INT_MIN: no such entry (one that is so is out of range anyway)
    return from < u_stop && e + lane < static_cast<uint32_t>(cnt) ? max(__ldg(a.sel + pair * a.capacity + e + lane), INT_MIN + 1) : INT_MIN;
  }
  __device__ __forceinline__ void load_page(int j, int& pg, int& rows) const {  // rows: valid rows of the page
    pg = rows = 0;
    if (j == INT_MIN) return;
    if (j < 0 || j >= min(ceil_div(max(L, 0), kv.block), kv.max_blocks)) {
      set_error(err, HS_EBIT_BLOCK_RANGE);
      return;
    }
    pg = __ldg(kv.page_table + pair * kv.max_blocks + j);
    if (pg < 0 || pg >= kv.num_pages) {
      set_error(err, HS_EBIT_PAGE_RANGE);
      pg = 0;
      return;
    }
    rows = min(kv.block, L - j * kv.block);
  }
  // Tiles [run0, run0 + tiles) of the first `count` selected blocks; `tokens` in the request.
  __device__ __forceinline__ TileRows(const KvView& view, const Args& args, int this_pair, int count, int tokens, int run0, int tiles,
                                      int this_lane, unsigned* error)
      : kv(view), a(args), err(error), pair(this_pair), lane(this_lane), cnt(count), L(tokens) {
    const uint32_t B = kv.block;
    u = static_cast<uint32_t>(run0) * kTile;
    u_stop = u + static_cast<uint32_t>(tiles) * kTile;
    e_base = u / B;
    j0 = load_sel(u, e_base);
    w_end = window_end(u, e_base);
    const uint32_t e1 = w_end / B;
    j1 = load_sel(w_end, e1);
    const uint32_t w_end1 = window_end(w_end, e1);
    j2 = load_sel(w_end1, w_end1 / B);
    load_page(j0, page, lim);
    load_page(j1, page1, lim1);
    ei = static_cast<int>((u + lane) / B);
    er = static_cast<int>(u + lane - ei * B);
    step_i = kTile / kv.block;
    step_r = kTile - step_i * kv.block;
  }
  // The lane's row of the next tile (0 where there is none); false: no such token.
  __device__ __forceinline__ bool next(uint32_t& row) {
    int place;
    return next_at<false>(row, place);
  }
  // With its place in the request.
  template <bool PLACE>
  __device__ __forceinline__ bool next_at(uint32_t& row, int& place) {
    if (u >= w_end) {  // the next window, whose pages are here; the pages of the one after it, whose entries are
      const uint32_t B = kv.block;
      e_base = w_end / B;
      w_end = window_end(w_end, e_base);
      page = page1;
      lim = lim1;
      if constexpr (PLACE) j0 = j1;
      load_page(j2, page1, lim1);
      if constexpr (PLACE) j1 = j2;
      const uint32_t w_end1 = window_end(w_end, w_end / B);
      j2 = load_sel(w_end1, w_end1 / B);
    }
    const int e = ei - static_cast<int>(e_base);
    if constexpr (PLACE) place = static_cast<int>(static_cast<uint32_t>(__shfl_sync(0xffffffffu, j0, e)) * static_cast<uint32_t>(kv.block)) + er;
    const int pg = __shfl_sync(0xffffffffu, page, e);
    const bool ok = er < __shfl_sync(0xffffffffu, lim, e);
    row = ok ? static_cast<uint32_t>(pg) * static_cast<uint32_t>(kv.block) + er : 0u;
    u += kTile;
    ei += step_i;
    er += step_r;
    if (er >= kv.block) {
      er -= kv.block;
      ++ei;
    }
    return ok;
  }
};

}  // namespace parts
}  // namespace
}  // namespace hs
