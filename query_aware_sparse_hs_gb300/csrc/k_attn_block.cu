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
// Work: the 32-token tiles of every (request, kv head)'s selection, from the
// actual counts, which every CTA sums; pairs are cut into equal parts for teams
// of warps (choose_cut below), and of a pair that is cut the team that arrives
// last merges the partial results in the parts' order (the same result whichever
// team that is).  The warps of a team take a run of the part's tiles each, with
// their own running maximum, sum and output, their own ring of tiles in shared
// memory filled by asynchronous 16-byte copies, and no barrier with the others
// until the part ends.
//
// Products on the warp-level matrix instruction m16n8k16 (f16 in, fp32 sums):
//   S[token][head] = K . Q^T: 16 tokens by 8 heads, so that the group of query
//     heads that shares the kv head fills the instruction's narrow side;
//   O^T[channel][head] += V^T . P^T: 16 channels by 8 heads over 16 tokens.
// (tcgen05 would take K's codes as they are, but P and V through shared and tensor
// memory: that chain, not the products, bounds the kernel of grouped scales at
// half the copy rate; here the matrix pipe is 23% busy, for uneven requests and for 16
// heads of 64 channels alike, and its e4m3 form of this instruction, which converts
// inside, was slower by an eighth.  A form whose V codes and P enter the 8-bit products
// of tcgen05 as they are has not been built.)
// Order of the contracted channels and of the output's channels is free, so a
// lane's operands are whole 16-byte pieces of a row as it lies in memory; V's
// transposition is one byte permutation per two operands.  Rows lie in shared
// memory with their 16-byte pieces XOR-permuted, so that neither reading order
// has bank conflicts.
//
// What bounds it: memory, for long work (16 requests x 4 heads x 131072 tokens, 2.15
// GB: 315 to 327 us from one GPU to another, 0.98 to 1.02 of the copy rate; 64
// channels 0.80).  Before it streams, a part waits for a chain of lookups (counts,
// selection, pages, rows: 4 us), after it for the join of its warps and, where pairs
// are cut, the merge (2 and 2 us): 32 requests x 4096 selected tokens, 134 MB, no pair
// cut: 28.8 us, 0.70.  (Asking the L2 ahead for selections and pages did not shorten
// the chain.)  With 16 query heads
// and 64 channels (12 requests x 2 heads, 75 MB: 31.0 us, 0.36) a 32-token tile takes an
// SM about 260 cycles whatever the number of warps, and about half of the call is
// start, join and merge of parts of ten tiles a warp.  (Codes converted by shifts on
// the integer pipe instead of the converting instruction, which retires 17 pairs a
// cycle: 3% slower; 64 tokens at a time: long runs 5% faster, 8% slower where a warp has
// few tiles.)  16 heads of 128 channels: 16 requests x 4 heads x 65536 tokens 228 us,
// 0.71; 255 registers, 56 bytes spilled.
//
// Precision: q times a power of two per head (largest entry into [256, 512)) is
// exact in f16 for entries within 2^-25 of the largest (eight bits down to 2^-24), and
// absolutely within 2^-33 of it below (half of 2^-24 in 256).  The power is 2^127 at
// most: a head whose largest entry is under 2^-118 is exact, as bf16 ends at 2^-133.
// P * vscale, in units of 2^-14 times the largest V scale met so far (a power of two,
// 2^-112 or more), enters as two f16 terms: 22 bits, and absolutely within 2^-25 of
// the units where it is under an eighth of them.  One term, for bf16 outputs, would
// save 2 to 3% with up to 8 heads (nothing where memory binds), 8% with 16 heads of 64
// channels and 20% of 128 (37.8 us for 47.0), and moves bf16 outputs by 6 10^-4 of
// their norm.  Sums, maxima and partial outputs are fp32; sums stay in those units
// until they are divided, so that V may be as large as its outputs can be.
#include <limits.h>

#include "attn_parts.cuh"

namespace hs {
namespace {

using namespace parts;

// Teams of a CTA, and with them the warps of an SM (one CTA on each): as many as
// the registers (128 channels: up to 255 a thread, 64 channels: 168) and the
// rings of tiles allow.  64 channels, 32 x 4 heads x 65536 tokens, with one term of P:
// 12 warps 195 us, 8 warps 222, 16 warps (128 registers) 192 but slower for short
// requests; with two terms 12 warps 202.
__host__ __device__ constexpr int teams_of(int head_dim) { return head_dim == 128 ? 2 : 3; }
constexpr int kStages = 3;      // tiles in a warp's ring

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
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

template <int D>
constexpr int ring_bytes() {
  return teams_of(D) * kTeamWarps * kStages * 2 * kTile * D;
}

template <int D, int NT>
__global__ __launch_bounds__(teams_of(D) * kTeamWarps * 32, 1) void attn_block_kernel(KvView kv, PartArgs a, unsigned* err) {
  constexpr int kTeams = teams_of(D), kWarps = kTeams * kTeamWarps;
  constexpr int kStageBytes = 2 * kTile * D;
  constexpr int kPieces = D / 16;        // 16-byte pieces of a row
  constexpr int kRowsPer = 32 / kPieces; // rows one copy instruction of a warp covers
  constexpr int kChunks = D / 64;        // 64-channel parts of a row (4 pieces each)
  extern __shared__ __align__(1024) uint8_t ring[];
  __shared__ float s_ks[kWarps][kStages][kTile], s_vs[kWarps][kStages][kTile];
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
  const int G = kv.group, B = kv.block;
  const int pairs = kv.batch * kv.hkv, ctas = gridDim.x;

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

  // this lane's 16-byte piece of the first rows a copy instruction covers
  const uint8_t* k_piece = static_cast<const uint8_t*>(kv.k_pages) + (lane / kPieces) * D + 16 * (lane % kPieces);
  const uint8_t* v_piece = static_cast<const uint8_t*>(kv.v_pages) + (lane / kPieces) * D + 16 * (lane % kPieces);
  uint8_t* my_ring = ring + warp * (kStages * kStageBytes);
  const uint32_t my_ring_addr = smem_addr(my_ring);

  const int my_parts = (all_parts - slot + cut.slots - 1) / cut.slots;
  for (int n_part = 0; n_part < my_parts; ++n_part) {
    if (n_part == listed + kListed) {
      listed = n_part;
      number_parts(kv, a, cut, team, s_scratch[tm], note);
    }
    // ---- the part: seg_tiles tiles of `pair` from seg0 on ----
    const Part part = s_parts[tm][n_part - listed];
    const int pair = part.pair;
    const int cnt = pair_count(a, pair);
    const int pair_tiles = tiles_of(kv, cnt), each = pair_tiles / part.count, more = pair_tiles - each * part.count;
    const int seg0 = part.index * each + min(part.index, more), seg_tiles = each + (part.index < more ? 1 : 0);
    const int ws_row = (part.row + part.index) * G;
    const int b = pair / kv.hkv, kvh = pair - b * kv.hkv;
    const int L = kv.seq_lens[b];
    const int nb = min(ceil_div(max(L, 0), B), kv.max_blocks);
    // the query's loads go out ahead of the rows'
    uint4 q_raw[NT][kChunks][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < kChunks; ++k) {
        q_raw[nt][k][0] = q_raw[nt][k][1] = make_uint4(0u, 0u, 0u, 0u);
        if (nt * 8 + g < G) {
          const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) +
                                                            (static_cast<int64_t>(b) * kv.hq + kvh * G + nt * 8 + g) * D + 64 * k + 16 * c4);
          q_raw[nt][k][0] = __ldg(src);
          q_raw[nt][k][1] = __ldg(src + 1);
        }
      }
    const int32_t* sel = a.sel + static_cast<int64_t>(pair) * a.capacity;
    const int32_t* table = kv.page_table + static_cast<int64_t>(pair) * kv.max_blocks;

    // The warp's tiles: a run of the part.
    const int run0 = seg0 + seg_tiles * team_warp / team.warps;
    const int tiles = seg0 + seg_tiles * (team_warp + 1) / team.warps - run0;
    // Selected blocks are looked up 32 at a time, one to a lane, the pages one
    // window ahead of the copies and the selection two, so that neither load is
    // waited for (looked up tile by tile, one tile ahead, 16-token pages took 458 us
    // where they now take 328).  A window holds the entries from that of its first tile on;
    // a tile that does not fit opens the next.
    const uint32_t u0 = static_cast<uint32_t>(run0) * kTile, u_stop = u0 + static_cast<uint32_t>(tiles) * kTile;
    const uint32_t Bu = B;
    const auto window_end = [&](uint32_t u, uint32_t e) {  // first token past the window's whole tiles
      return u + ((e + 32) * Bu - u) / kTile * kTile;
    };
    const auto load_sel = [&](uint32_t u, uint32_t e) {  // INT_MIN: no such entry (one that is INT_MIN is out of range anyway)
      return u < u_stop && e + lane < static_cast<uint32_t>(cnt) ? max(__ldg(sel + e + lane), INT_MIN + 1) : INT_MIN;
    };
    const auto load_page = [&](int j, int& page, int& lim) {  // lim: valid rows of the page
      page = lim = 0;
      if (j == INT_MIN) return;
      if (j < 0 || j >= nb) {
        set_error(err, HS_EBIT_BLOCK_RANGE);
        return;
      }
      page = __ldg(table + j);
      if (page < 0 || page >= kv.num_pages) {
        set_error(err, HS_EBIT_PAGE_RANGE);
        page = 0;
        return;
      }
      lim = min(B, L - j * B);
    };
    uint32_t w_end, w_end1, w_end2;  // of the window in use, the next, the one after
    uint32_t e_base = u0 / Bu, e1, e2;
    int page, lim, page1, lim1, j2;
    {
      const int j0 = load_sel(u0, e_base);
      w_end = window_end(u0, e_base);
      e1 = w_end / Bu;
      const int j1 = load_sel(w_end, e1);
      w_end1 = window_end(w_end, e1);
      e2 = w_end1 / Bu;
      j2 = load_sel(w_end1, e2);
      w_end2 = window_end(w_end1, e2);
      load_page(j0, page, lim);
      load_page(j1, page1, lim1);
    }
    // this lane's row of the next tile: its entry and its row in the block
    uint32_t u = u0;
    int ei = static_cast<int>((u0 + lane) / Bu), er = static_cast<int>(u0 + lane - ei * Bu);
    const int step_i = kTile / B, step_r = kTile - step_i * B;
    int stage_in = 0;
    const auto issue = [&]() {  // the copies of the next tile
      if (u >= w_end) {
        e_base = e1;
        w_end = w_end1;
        page = page1;
        lim = lim1;
        e1 = e2;
        w_end1 = w_end2;
        load_page(j2, page1, lim1);
        e2 = w_end2 / Bu;
        j2 = load_sel(w_end2, e2);
        w_end2 = window_end(w_end2, e2);
      }
      const int pg = __shfl_sync(0xffffffffu, page, ei - static_cast<int>(e_base));
      const bool ok = er < __shfl_sync(0xffffffffu, lim, ei - static_cast<int>(e_base));
      const uint32_t live = __ballot_sync(0xffffffffu, ok);
      const uint32_t row = ok ? static_cast<uint32_t>(pg) * B + er : 0u;
      const uint32_t dst = my_ring_addr + stage_in * kStageBytes;
      if (live == 0xffffffffu && (B & 15) == 0) {  // 16 rows in a row of one page, twice
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint64_t at = static_cast<uint64_t>(__shfl_sync(0xffffffffu, row, 16 * h)) * D;
          const uint8_t* ks = k_piece + at;
          const uint8_t* vs = v_piece + at;
#pragma unroll
          for (int i = 0; i < 16 / kRowsPer; ++i) {
            const int r = 16 * h + i * kRowsPer + lane / kPieces;
            copy16(dst + piece_at<D>(r, lane % kPieces), ks + i * kRowsPer * D);
            copy16(dst + kTile * D + piece_at<D>(r, lane % kPieces), vs + i * kRowsPer * D);
          }
        }
      } else {  // any rows; those that are not there are zeros
#pragma unroll
        for (int i = 0; i < kTile / kRowsPer; ++i) {
          const int r = i * kRowsPer + lane / kPieces;
          const uint64_t at = static_cast<uint64_t>(__shfl_sync(0xffffffffu, row, r)) * D - (lane / kPieces) * D;
          const bool there = (live >> r) & 1u;
          copy16_if(dst + piece_at<D>(r, lane % kPieces), k_piece + at, there);
          copy16_if(dst + kTile * D + piece_at<D>(r, lane % kPieces), v_piece + at, there);
        }
      }
      copy4(smem_addr(&s_ks[warp][stage_in][lane]), kv.k_scales + pg, ok);
      copy4(smem_addr(&s_vs[warp][stage_in][lane]), kv.v_scales + pg, ok);
      if (lane == 0) s_live[warp][stage_in] = live;
      stage_in = stage_in + 1 == kStages ? 0 : stage_in + 1;
      u += kTile;
      ei += step_i;
      er += step_r;
      if (er >= B) {
        er -= B;
        ++ei;
      }
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

    // ---- the query, as the S product's second operand ----
    uint32_t qf[NT][4 * kChunks][2];
    float qs[NT][2];  // logit factor of heads 2 c4, 2 c4 + 1 (log2 units)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float x[kChunks][16];
      float amax = 0.0f;
#pragma unroll
      for (int k = 0; k < kChunks; ++k) {
        const uint4 v0 = q_raw[nt][k][0], v1 = q_raw[nt][k][1];
        const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[k][2 * i] = __uint_as_float(w[i] << 16);
          x[k][2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
          amax = fmaxf(amax, fmaxf(fabsf(x[k][2 * i]), fabsf(x[k][2 * i + 1])));
        }
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      float f = 1.0f;  // 2^(8 - exponent of amax), 2^127 at most
      if (amax > 0.0f && amax < INFINITY) f = __uint_as_float(static_cast<uint32_t>(min(254, 262 - static_cast<int>(__float_as_uint(amax) >> 23))) << 23);
      const float fs = a.scale < 0.0f ? -f : f;  // the factors of the logits are not negative
#pragma unroll
      for (int k = 0; k < kChunks; ++k)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          qf[nt][4 * k + w][0] = pack_half2(x[k][4 * w] * fs, x[k][4 * w + 1] * fs);
          qf[nt][4 * k + w][1] = pack_half2(x[k][4 * w + 2] * fs, x[k][4 * w + 3] * fs);
        }
      // (times -inf is -inf, for a scale of 0 too: 2^-149, and no logit passes 2^127)
      const float s = fmaxf(fabsf(a.scale) * kLog2e / f, __uint_as_float(1u));
      qs[nt][0] = __shfl_sync(0xffffffffu, s, 8 * c4);
      qs[nt][1] = __shfl_sync(0xffffffffu, s, 8 * c4 + 4);
    }

    float m[NT][2], l[NT][2];
    float base[NT][2];  // the maximum, 0 as long as there is none
    float o[NT][D / 16][4];
    float vref = kMinRef;  // power of two, not below the V scales met
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      base[nt][0] = base[nt][1] = 0.0f;
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
      copies_wait<kStages - 1>();
      __syncwarp();
      const uint8_t* kt = my_ring + stage * kStageBytes;
      const uint8_t* vt = kt + kTile * D;
      const float* ks = s_ks[warp][stage];
      const float* vs = s_vs[warp][stage];
      const uint32_t live = s_live[warp][stage];

      // S = K Q^T, the two 16-token halves in turn so that no product waits for the last
      float s[2][NT][4];
#pragma unroll
      for (int st = 0; st < 2; ++st)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[st][nt][e] = 0.0f;
#pragma unroll
      for (int k = 0; k < kChunks; ++k) {
        uint32_t wa[2][4], wb[2][4];
#pragma unroll
        for (int st = 0; st < 2; ++st) {
          const int ra = 16 * st + token_of<D>(g);
          const uint4 xa = *reinterpret_cast<const uint4*>(kt + piece_at<D>(ra, 4 * k + c4));
          const uint4 xb = *reinterpret_cast<const uint4*>(kt + piece_at<D>(ra + 8, 4 * k + c4));
          wa[st][0] = xa.x; wa[st][1] = xa.y; wa[st][2] = xa.z; wa[st][3] = xa.w;
          wb[st][0] = xb.x; wb[st][1] = xb.y; wb[st][2] = xb.z; wb[st][3] = xb.w;
        }
#pragma unroll
        for (int w = 0; w < 4; ++w)
#pragma unroll
          for (int st = 0; st < 2; ++st) {
            uint32_t a0, a1, a2, a3;
            e4m3x4_to_halves(wa[st][w], a0, a2);
            e4m3x4_to_halves(wb[st][w], a1, a3);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma(s[st][nt], a0, a1, a2, a3, qf[nt][4 * k + w][0], qf[nt][4 * k + w][1]);
          }
      }

      // logits (log2 units), their maximum over the tile
      float kr[4], vr[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 8 * i + token_of<D>(g);
        kr[i] = ks[r];
        vr[i] = vs[r];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          s[i >> 1][nt][2 * (i & 1)] *= kr[i];  // (times qs: the logit)
          s[i >> 1][nt][2 * (i & 1) + 1] *= kr[i];
        }
      }
      if (live != 0xffffffffu) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (!((live >> (8 * i + token_of<D>(g))) & 1u)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) s[i >> 1][nt][2 * (i & 1)] = s[i >> 1][nt][2 * (i & 1) + 1] = -INFINITY;
          }
      }
      bool raised = false;
      float mn[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float top = -INFINITY;
#pragma unroll
          for (int i = 0; i < 4; ++i) top = fmaxf(top, s[i >> 1][nt][2 * (i & 1) + e]);
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
          mn[nt][e] = fmaxf(m[nt][e], top * qs[nt][e]);
          raised |= mn[nt][e] > m[nt][e];
        }
      const uint32_t vmax = __reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(vs[lane])));
      const uint32_t vcap = max(__float_as_uint(vref), min((vmax + 0x7fffffu) & 0x7f800000u, kMaxRef));
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
            base[nt][e] = mn[nt][e] == -INFINITY ? 0.0f : mn[nt][e];
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              o[nt][i][e] *= f * down;
              o[nt][i][2 + e] *= f * down;
            }
          }
      }
      const float unit = unit_over(vref);
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
              p[e] = exp2_fast(fmaf(s[st][nt][2 * i + e], qs[nt][e], -base[nt][e]));
              l[nt][e] += p[e];
              p[e] *= vr[2 * st + i];
            }
            const uint32_t hi = pack_half2(p[0], p[1]);
            ph[nt][i] = transpose8x8(hi);
            const float2 back = unpack_half2(hi);
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
          uint32_t a0, a1, a2, a3;
          e4m3x4_to_halves(y0, a0, a1);
          e4m3x4_to_halves(y1, a2, a3);
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
    team.sync();  // every warp is done with its ring: the team's rings now hold the outputs
    if (lane == 0) s_ref[warp] = vref;
    float* so = reinterpret_cast<float*>(ring + first_warp * (kStages * kStageBytes));  // [team warp][8 NT][D]
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
        float* dst = so + (team_warp * 8 * NT + h) * D + g * (D / 8);
#pragma unroll
        for (int i = 0; i < D / 16; i += 2)
          *reinterpret_cast<float4*>(dst + 2 * i) =
              make_float4(o[nt][i][e], o[nt][i][2 + e], o[nt][i + 1][e], o[nt][i + 1][2 + e]);
      }
    team.sync();
    finish_part<D, NT>(kv, a, team, part, s_m + first_warp, s_l + first_warp, s_ref + first_warp, so, &s_last[tm]);
    team.sync();  // the rings and s_m are free again
  }
}

template <int D, int NT>
cudaError_t launch_n(const KvView& kv, const PartArgs& b, int ctas, unsigned* err, cudaStream_t st) {
  auto kern = attn_block_kernel<D, NT>;
  static std::atomic<uint64_t> allowed{0};
  if (cudaError_t e = allow_dynamic_smem_once(allowed, kern, ring_bytes<D>()); e != cudaSuccess) return e;
  cudaError_t e = launch_pdl(kern, dim3(ctas), dim3(teams_of(D) * kTeamWarps * 32), ring_bytes<D>(), st, kv, b, err);
  if (e != cudaSuccess || b.counters) return e;
  const size_t smem = (static_cast<size_t>(ctas * teams_of(D) + 2) * kv.group + 4 +
                       static_cast<size_t>(teams_of(D) - 1) * kv.group * D) * sizeof(float);
  auto merge = merge_parts_kernel<D, NT, teams_of(D)>;
  if ((e = allow_dynamic_smem(merge, smem)) != cudaSuccess) return e;
  return launch_pdl(merge, dim3(kv.batch * kv.hkv), dim3(teams_of(D) * kTeamWarps * 32), smem, st, kv, b, ctas);
}

}  // namespace

int block_attn_rows(int ctas, int head_dim) { return 2 * ctas * teams_of(head_dim); }

cudaError_t launch_block_attn(const KvView& kv, const AttnArgs& a, unsigned* err, cudaStream_t st) {
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
  const int ctas = a.sms;
  if (kv.head_dim == 128)
    return kv.group <= 8 ? launch_n<128, 1>(kv, b, ctas, err, st) : launch_n<128, 2>(kv, b, ctas, err, st);
  return kv.group <= 8 ? launch_n<64, 1>(kv, b, ctas, err, st) : launch_n<64, 2>(kv, b, ctas, err, st);
}

}  // namespace hs
