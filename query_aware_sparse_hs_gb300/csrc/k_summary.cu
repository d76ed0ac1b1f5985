// Per-block key summaries (Quest, "KV 稀疏化" wiki §5): channel-wise min and
// max of K over each block's valid tokens.  Each lane owns 16 bytes of
// consecutive channels of a row, so one warp load reads whole consecutive
// rows.  HBM-bound: one pass over the K pages of the blocks asked for.
#include "hs_internal.h"
#include "int4.cuh"

namespace hs {
namespace {

// Each lane loads 16 bytes of a row (V channels), so a warp load covers RPL
// consecutive rows of the page - one contiguous 512-byte span - and a lane
// keeps U loads in flight before it uses any.
template <int KIND>
struct Elem;
template <>
struct Elem<HS_KV_F32> { static constexpr int kBytes = 4; };
template <>
struct Elem<HS_KV_BF16> { static constexpr int kBytes = 2; };
template <>
struct Elem<HS_KV_FP8E4M3_G32> { static constexpr int kBytes = 1; };

// 16 bytes of one row -> min/max of its V channels into mn/mx
template <int KIND, int V>
__device__ __forceinline__ void fold(const uint4& raw, float s, float (&mn)[V], float (&mx)[V]) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  if constexpr (KIND == HS_KV_F32) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float x = __uint_as_float(w[c]);
      mn[c] = fminf(mn[c], x); mx[c] = fmaxf(mx[c], x);
    }
  } else if constexpr (KIND == HS_KV_BF16) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float lo = __uint_as_float(w[c] << 16), hi = __uint_as_float(w[c] & 0xffff0000u);
      mn[2 * c] = fminf(mn[2 * c], lo); mx[2 * c] = fmaxf(mx[2 * c], lo);
      mn[2 * c + 1] = fminf(mn[2 * c + 1], hi); mx[2 * c + 1] = fmaxf(mx[2 * c + 1], hi);
    }
  } else {
    // e4m3 K: code value times the token's 32-channel group scale, in fp32
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const float2 x = e4m3x2_to_float2(static_cast<uint16_t>(w[c >> 1] >> (16 * (c & 1))));
      const float a = x.x * s, b = x.y * s;
      mn[2 * c] = fminf(mn[2 * c], a); mx[2 * c] = fmaxf(mx[2 * c], a);
      mn[2 * c + 1] = fminf(mn[2 * c + 1], b); mx[2 * c + 1] = fmaxf(mx[2 * c + 1], b);
    }
  }
}

constexpr int kWarps = 8;

// Warps per block: enough that each warp reads about one round of R rows per
// block (from 1 to 8); a CTA of 8 warps covers 8 / wpb blocks, and the warps'
// partial boxes are combined in shared memory.
__host__ __device__ __forceinline__ int warps_per_block(int B, int R) { return B >= 8 * R ? 8 : (B >= R ? B / R : 1); }

// rows in flight per lane: up to 8, no more than a block holds per warp load
__host__ __forceinline__ int rounds_for(int B, int rpl) {
  const int r = ceil_div(B, rpl);
  return r >= 8 ? 8 : (r >= 4 ? 4 : (r >= 2 ? 2 : 1));
}

// Persistent: CTA x takes block groups x, x + gridDim.x, ... of the flattened
// (request, kv head, group of per_cta blocks) space; groups past a request's
// blocks are skipped without work (requests of very different lengths would
// otherwise launch most CTAs for nothing).
template <int D, int KIND, int U>
__global__ __launch_bounds__(kWarps * 32) void summaries_kernel(KvView kv, int first_block, int groups_per_pair,
                                                               int64_t total_groups, void* smin, void* smax,
                                                               unsigned* err) {
  constexpr int E = Elem<KIND>::kBytes, V = 16 / E, LPR = D / V, RPL = 32 / LPR, R = RPL * U;
  static_assert(D % V == 0 && 32 % LPR == 0, "a row is a whole number of 16-byte lanes");
  __shared__ float s_mn[kWarps][D], s_mx[kWarps][D];
  __shared__ int s_ok[kWarps];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rs = lane / LPR, d0 = (lane % LPR) * V;
  const int B = kv.block;
  const int wpb = warps_per_block(B, R), per_cta = kWarps / wpb;
  const int bl = warp / wpb, sub = warp % wpb;
  for (int64_t gi = blockIdx.x; gi < total_groups; gi += gridDim.x) {
    const int64_t pair = gi / groups_per_pair;
    const int grp = static_cast<int>(gi - pair * groups_per_pair);
    const int b = static_cast<int>(pair / kv.hkv);
    const int L = kv.seq_lens[b];
    const int nb = min(ceil_div(max(L, 0), B), kv.max_blocks);
    const int jg = first_block + grp * per_cta;  // the group's first block
    if (jg >= nb) continue;  // the same for every thread of the CTA
    const int j = jg + bl;
    float mn[V], mx[V];
#pragma unroll
    for (int c = 0; c < V; ++c) { mn[c] = INFINITY; mx[c] = -INFINITY; }
    bool ok = bl < per_cta && j < nb;
    if (ok) {
      const int page = kv.page_table[pair * kv.max_blocks + j];
      if (page < 0 || page >= kv.num_pages) {
        if (lane == 0 && sub == 0) set_error(err, HS_EBIT_PAGE_RANGE);
        ok = false;
      } else {
        const int valid = min(B, L - j * B);
        const int64_t row0 = static_cast<int64_t>(page) * B;
        const uint8_t* base = static_cast<const uint8_t*>(kv.k_pages) + d0 * E;
        for (int t0 = sub * RPL; t0 < valid; t0 += wpb * R) {
          uint4 raw[U];
          float sc[U];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            // clamp: a repeated valid row changes nothing
            const int64_t row = row0 + min(t0 + u * wpb * RPL + rs, valid - 1);
            raw[u] = __ldg(reinterpret_cast<const uint4*>(base + row * (D * E)));
            if constexpr (KIND == HS_KV_FP8E4M3_G32)
              sc[u] = __ldg(kv.k_scales + row * (D / kQuantGroup) + d0 / kQuantGroup);
            else
              sc[u] = 1.0f;
          }
#pragma unroll
          for (int u = 0; u < U; ++u) fold<KIND, V>(raw[u], sc[u], mn, mx);
        }
      }
    }
    // the RPL row slots of the warp hold the same channels: combine them
#pragma unroll
    for (int off = LPR; off < 32; off <<= 1)
#pragma unroll
      for (int c = 0; c < V; ++c) {
        mn[c] = fminf(mn[c], __shfl_xor_sync(0xffffffffu, mn[c], off));
        mx[c] = fmaxf(mx[c], __shfl_xor_sync(0xffffffffu, mx[c], off));
      }
    if (rs == 0)
#pragma unroll
      for (int c = 0; c < V; ++c) { s_mn[warp][d0 + c] = mn[c]; s_mx[warp][d0 + c] = mx[c]; }
    if (lane == 0) s_ok[warp] = ok ? 1 : 0;
    __syncthreads();
    for (int idx = threadIdx.x; idx < per_cta * D; idx += kWarps * 32) {
      const int cb = idx / D, d = idx - cb * D;
      const int w0 = cb * wpb;
      if (!s_ok[w0]) continue;
      float lo = s_mn[w0][d], hi = s_mx[w0][d];
      for (int w = 1; w < wpb; ++w) { lo = fminf(lo, s_mn[w0 + w][d]); hi = fmaxf(hi, s_mx[w0 + w][d]); }
      const int64_t o = (pair * kv.max_blocks + jg + cb) * D + d;
      if constexpr (KIND == HS_KV_F32) {
        static_cast<float*>(smin)[o] = lo;
        static_cast<float*>(smax)[o] = hi;
      } else {
        // bf16 K: min/max are bf16 values, the conversion is exact.  e4m3 K:
        // round outward so the stored box still contains every dequantised key.
        static_cast<__nv_bfloat16*>(smin)[o] = (KIND == HS_KV_BF16) ? __float2bfloat16_rn(lo) : __float2bfloat16_rd(lo);
        static_cast<__nv_bfloat16*>(smax)[o] = (KIND == HS_KV_BF16) ? __float2bfloat16_rn(hi) : __float2bfloat16_ru(hi);
      }
    }
    __syncthreads();  // the shared buffers are reused by the next group
  }
}

template <int D, int KIND, int U>
cudaError_t launch_u(const KvView& kv, int first_block, int nblocks, void* smin, void* smax,
                     unsigned* err, int sms, cudaStream_t st) {
  constexpr int RPL = 32 / (D * Elem<KIND>::kBytes / 16);
  const int per_cta = kWarps / warps_per_block(kv.block, RPL * U);
  const int gpp = ceil_div(nblocks, per_cta);
  const int64_t total = static_cast<int64_t>(gpp) * kv.hkv * kv.batch;
  static int per_sm = 0;  // resident CTAs of this kernel per SM
  if (per_sm == 0) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, summaries_kernel<D, KIND, U>, kWarps * 32, 0) !=
            cudaSuccess ||
        per_sm < 1)
      per_sm = 1;
  }
  const int64_t resident = static_cast<int64_t>(sms > 0 ? sms : 148) * per_sm;
  const unsigned grid = static_cast<unsigned>(total < resident ? total : resident);
  return launch_pdl(summaries_kernel<D, KIND, U>, dim3(grid), dim3(kWarps * 32), 0, st, kv, first_block, gpp, total,
                    smin, smax, err);
}

template <int D, int KIND>
cudaError_t launch_k(const KvView& kv, int first_block, int nblocks, void* smin, void* smax,
                     unsigned* err, int sms, cudaStream_t st) {
  constexpr int RPL = 32 / (D * Elem<KIND>::kBytes / 16);
  switch (rounds_for(kv.block, RPL)) {
    case 8: return launch_u<D, KIND, 8>(kv, first_block, nblocks, smin, smax, err, sms, st);
    case 4: return launch_u<D, KIND, 4>(kv, first_block, nblocks, smin, smax, err, sms, st);
    case 2: return launch_u<D, KIND, 2>(kv, first_block, nblocks, smin, smax, err, sms, st);
    default: return launch_u<D, KIND, 1>(kv, first_block, nblocks, smin, smax, err, sms, st);
  }
}

// A warp's equal run of the blocks of all requests and kv heads, end to end.  All 32
// lanes call the constructor; `w` of `warps` warps.
struct BlockRun {
  const KvView& kv;
  int first_block, req, n_req, j;  // the request, its blocks, the block
  int64_t pair, g, g_end;

  __device__ __forceinline__ int blocks_of(int b) const {
    return max(min(ceil_div(max(__ldg(kv.seq_lens + b), 0), kv.block), kv.max_blocks) - first_block, 0);
  }
  __device__ __forceinline__ BlockRun(const KvView& view, int first, int64_t w, int64_t warps, int lane)
      : kv(view), first_block(first), req(0), n_req(0), j(0), pair(0) {
    const int batch = kv.batch, mine_n = (batch + 31) / 32, b0 = min(batch, lane * mine_n), b1 = min(batch, b0 + mine_n);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) mine += blocks_of(b);
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const int64_t total = __shfl_sync(0xffffffffu, incl, 31) * kv.hkv;
    const int64_t per = (total + warps - 1) / warps;
    g = w * per;
    g_end = min(total, g + per);
    if (g >= g_end) return;
    int64_t before = 0;  // blocks of the requests before req, all kv heads
    const unsigned has = __ballot_sync(0xffffffffu, incl * kv.hkv > g);
    const int owner = __ffs(has) - 1;
    if (lane == owner) {
      before = (incl - mine) * kv.hkv;
      for (req = b0; req < b1 - 1; ++req) {
        const int64_t n = static_cast<int64_t>(blocks_of(req)) * kv.hkv;
        if (g < before + n) break;
        before += n;
      }
    }
    req = __shfl_sync(0xffffffffu, req, owner);
    before = __shfl_sync(0xffffffffu, before, owner);
    n_req = blocks_of(req);
    pair = static_cast<int64_t>(req) * kv.hkv + (g - before) / n_req;
    j = first_block + static_cast<int>((g - before) % n_req);
  }
  __device__ __forceinline__ bool more() const { return g < g_end; }
  // Blocks from j on that are of the same pair and this run's, 32 at most.
  __device__ __forceinline__ int count() const {
    return static_cast<int>(min(static_cast<int64_t>(min(32, first_block + n_req - j)), g_end - g));
  }
  __device__ __forceinline__ void on(int n) {
    g += n;
    j += n;
    if (j < first_block + n_req) return;
    j = first_block;
    ++pair;
    if (pair == static_cast<int64_t>(req + 1) * kv.hkv && g < g_end) {
      do {  // the next request with blocks: there is one before g_end
        ++req;
        n_req = blocks_of(req);
      } while (n_req == 0);
      pair = static_cast<int64_t>(req) * kv.hkv;
    }
  }
};

// ---- e4m3 with one scale per page ----
// The scale is the same for the whole block, so min and max are taken over the
// codes, as f16 pairs (which hold every e4m3 number), and only the two results
// are scaled: 2 conversions and 4 two-wide comparisons for 4 codes, where the
// grouped kind needs 4 products and 8 comparisons more.  A lane owns 4
// neighbouring channels of every row it loads, so the block needs no exchange
// between lanes (64 channels: one with the other half of the warp), and a warp
// none with other warps.  The blocks of all requests and kv heads are laid end to
// end and cut into equal runs, one per warp (every warp sums the requests' block
// counts); a warp looks up 32 blocks of its run together and loads the next 16
// rows (64 channels: 32; half as many for short blocks) while it folds the last.
// Memory-bound: 32 requests x 4 heads of 4K to 64K tokens, 16-token pages of 128
// channels, 770 MB: 128 us, 0.90 of the copy rate (the common kernel above: 400).
__device__ __forceinline__ void codes_to_half2(uint32_t w, __half2& a, __half2& b) {
  uint32_t x, y;
  e4m3x4_to_halves(w, x, y);
  a = *reinterpret_cast<__half2*>(&x);
  b = *reinterpret_cast<__half2*>(&y);
}
__device__ __forceinline__ __half2 shfl_half2(__half2 v, int off) {
  const uint32_t x = __shfl_xor_sync(0xffffffffu, *reinterpret_cast<uint32_t*>(&v), off);
  return *reinterpret_cast<const __half2*>(&x);
}

// Loads in flight: 16, or 8 where those are a whole block (64 channels, 16-token
// pages: 78 us, with 16 loads, half of them repeats, 112).  CTAs per SM: as the
// registers allow.
constexpr int block_ctas(int rows) { return rows == 16 ? 3 : 5; }

template <int D, int kRows>
__global__ __launch_bounds__(kWarps * 32, block_ctas(kRows)) void summaries_block_kernel(KvView kv, int first_block, void* smin,
                                                                                 void* smax, unsigned* err) {
  constexpr int RPL = 128 / D;  // rows of one warp load
  constexpr int kStep = kRows * RPL;
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int rs = lane / (D / 4), d0 = lane % (D / 4) * 4;
  const int B = kv.block;
  BlockRun run(kv, first_block, static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5),
               static_cast<int64_t>(gridDim.x) * kWarps, lane);
  while (run.more()) {
    // ---- up to 32 blocks of one pair ----
    const int n = run.count(), j = run.j;
    const int64_t pair = run.pair;
    const int L = __ldg(kv.seq_lens + run.req);
    int my_page = -1;
    float my_scale = 0.0f;
    if (lane < n) {
      my_page = __ldg(kv.page_table + pair * kv.max_blocks + j + lane);
      if (my_page < 0 || my_page >= kv.num_pages) {
        set_error(err, HS_EBIT_PAGE_RANGE);
        my_page = -1;
      } else {
        my_scale = __ldg(kv.k_scales + my_page);
      }
    }
    unsigned left = __ballot_sync(0xffffffffu, my_page >= 0);
    uint32_t raw[kRows], next[kRows];
    const auto load = [&](uint32_t (&r)[kRows], int i, int t0) {
      const int page = __shfl_sync(0xffffffffu, my_page, i);
      const int last = min(B, L - (j + i) * B) - 1;
      const uint8_t* base = static_cast<const uint8_t*>(kv.k_pages) + static_cast<int64_t>(page) * B * D + d0;
#pragma unroll
      for (int u = 0; u < kRows; ++u)  // clamp: a repeated valid row changes nothing
        r[u] = __ldg(reinterpret_cast<const uint32_t*>(base + min(t0 + u * RPL + rs, last) * D));
    };
    __half2 mn[2], mx[2];
    mn[0] = mn[1] = __half2half2(__ushort_as_half(0x7c00));  // inf
    mx[0] = mx[1] = __half2half2(__ushort_as_half(0xfc00));
    int i = left ? __ffs(left) - 1 : 32, t0 = 0;
    if (left) load(next, i, 0);
    while (left) {
#pragma unroll
      for (int u = 0; u < kRows; ++u) raw[u] = next[u];
      const int now = i;
      const bool ends = t0 + kStep >= min(B, L - (j + i) * B);
      if (ends) {
        left &= left - 1;
        i = left ? __ffs(left) - 1 : 32;
        t0 = 0;
      } else {
        t0 += kStep;
      }
      if (left) load(next, i, t0);
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        __half2 x, y;
        codes_to_half2(raw[u], x, y);
        mn[0] = __hmin2(mn[0], x);
        mn[1] = __hmin2(mn[1], y);
        mx[0] = __hmax2(mx[0], x);
        mx[1] = __hmax2(mx[1], y);
      }
      if (ends) {
        const float scale = __shfl_sync(0xffffffffu, my_scale, now);
        if constexpr (RPL > 1)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            mn[c] = __hmin2(mn[c], shfl_half2(mn[c], 16));
            mx[c] = __hmax2(mx[c], shfl_half2(mx[c], 16));
          }
        if (rs == 0) {
          const int64_t o = (pair * kv.max_blocks + j + now) * D + d0;
          __nv_bfloat162 lo[2], hi[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {  // outward: the stored box still contains every dequantised key
            const float2 x = __half22float2(mn[c]), y = __half22float2(mx[c]);
            lo[c].x = __float2bfloat16_rd(x.x * scale);
            lo[c].y = __float2bfloat16_rd(x.y * scale);
            hi[c].x = __float2bfloat16_ru(y.x * scale);
            hi[c].y = __float2bfloat16_ru(y.y * scale);
          }
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(smin) + o) = *reinterpret_cast<const uint2*>(lo);
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(smax) + o) = *reinterpret_cast<const uint2*>(hi);
        }
        mn[0] = mn[1] = __half2half2(__ushort_as_half(0x7c00));
        mx[0] = mx[1] = __half2half2(__ushort_as_half(0xfc00));
      }
    }
    run.on(n);
  }
}

template <int D, int kRows>
cudaError_t launch_block_rows(const KvView& kv, int first_block, int nblocks, void* smin, void* smax, unsigned* err,
                              int sms, cudaStream_t st) {
  // a warp for each block at most
  const int64_t most = (static_cast<int64_t>(kv.batch) * kv.hkv * nblocks + kWarps - 1) / kWarps;
  const int resident = sms * block_ctas(kRows);
  const unsigned grid = static_cast<unsigned>(most < resident ? most : resident);
  return launch_pdl(summaries_block_kernel<D, kRows>, dim3(grid), dim3(kWarps * 32), 0, st, kv, first_block, smin, smax,
                    err);
}

template <int D>
cudaError_t launch_block(const KvView& kv, int first_block, int nblocks, void* smin, void* smax, unsigned* err,
                         int sms, cudaStream_t st) {
  return kv.block <= 8 * (128 / D) ? launch_block_rows<D, 8>(kv, first_block, nblocks, smin, smax, err, sms, st)
                                   : launch_block_rows<D, 16>(kv, first_block, nblocks, smin, smax, err, sms, st);
}

// ---- 4-bit codes ----
// Every row has scales and centres of its own, so each value is formed in fp32
// (z + s c) before it is compared.  A lane owns 8 neighbouring channels, which are of
// one group, a warp a run of blocks; a block's row slots are joined by halving the
// channels.  A code becomes a number by masking its bits where they are (8 ors and masks,
// one shift: 2^23 + 16^i n), one addition and one fused multiply of two at a time, its
// scale being s / 16^i.
// What bounds it: instructions, two thirds of them comparisons, masks and shifts, whose
// pipe is busy for two thirds of the time.  32 requests x 4 heads of 4K to 64K tokens,
// 128 channels: 138 us with 64-token pages (0.45 of the copy rate), 161 with 16-token pages
// (0.49); full units without a clamp of the rows: 152 and 175 with it.  (Before that, 16
// channels to a lane: 148 and 190 us; additions and multiplies one at a time 155 and 177;
// rows loaded into registers instead of the ring 162 and 201.)
__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy8_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
// 2^23 + n 16^i: the code's bits where they are, below the exponent of 2^23 (`magic`, in
// a register).
template <uint32_t MASK>
__device__ __forceinline__ float number(uint32_t v, uint32_t magic) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(v), "n"(MASK), "r"(magic));  // (v & MASK) | magic
  return __uint_as_float(d);
}
// 8 channels of a row as they lie in memory.
struct Codes8 {
  uint32_t w;
  uint32_t s, z;  // in the low half
  // What they stand for.
  __device__ __forceinline__ void get(float (&x)[8], uint32_t magic) const {
    const float f = __uint_as_float(s << 16), c = __uint_as_float(z << 16);
    const float f1 = f * 0.0625f, f2 = f * 0.00390625f, f3 = f * 0.000244140625f, f4 = f * 0.0000152587890625f;
    constexpr float k = 8388608.0f;  // 2^23
    const float2 centre = make_float2(c, c);
    const uint32_t lo = w, up = w >> 20;
    const float2 a = int4::add_pair(make_float2(number<0xfu>(lo, magic), number<0xf0u>(lo, magic)), make_float2(-k - 8.0f, -k - 128.0f));
    const float2 b = int4::add_pair(make_float2(number<0xf00u>(lo, magic), number<0xf000u>(lo, magic)), make_float2(-k - 2048.0f, -k - 32768.0f));
    const float2 d = int4::add_pair(make_float2(number<0xf0000u>(lo, magic), number<0xfu>(up, magic)), make_float2(-k - 524288.0f, -k - 8.0f));
    const float2 e = int4::add_pair(make_float2(number<0xf0u>(up, magic), number<0xf00u>(up, magic)), make_float2(-k - 128.0f, -k - 2048.0f));
    const float2 va = int4::fma_pair(a, make_float2(f, f1), centre), vb = int4::fma_pair(b, make_float2(f2, f3), centre);
    const float2 vd = int4::fma_pair(d, make_float2(f4, f), centre), ve = int4::fma_pair(e, make_float2(f1, f2), centre);
    x[0] = va.x; x[1] = va.y; x[2] = vb.x; x[3] = vb.y;
    x[4] = vd.x; x[5] = vd.y; x[6] = ve.x; x[7] = ve.y;
  }
};

// A warp's rows go through its ring in shared memory in units of up to 16 rows of a
// block, kUnits - 1 of them on their way.
constexpr int kUnitRows = 16, kUnits = 6;
template <int D>
struct Unit {
  static constexpr int kCodes = kUnitRows * int4::row_bytes(D), kBytes = kCodes + kUnitRows * int4::record(D) * 2;
};

template <int D>
__global__ __launch_bounds__(kWarps * 32, 3) void summaries_int4_kernel(KvView kv, int first_block, void* smin, void* smax,
                                                                        unsigned* err) {
  constexpr int LPR = D / 8, RPL = 32 / LPR;  // lanes of a row, rows of a warp at a time
  constexpr int kRecord = int4::record(D) * 2;
  extern __shared__ __align__(128) uint8_t ring[];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rs = lane / LPR, d0 = lane % LPR * 8;
  const int B = kv.block;
  uint8_t* mine = ring + warp * (kUnits * Unit<D>::kBytes);
  const uint32_t mine_addr = static_cast<uint32_t>(__cvta_generic_to_shared(mine));
  BlockRun run(kv, first_block, static_cast<int64_t>(blockIdx.x) * kWarps + warp, static_cast<int64_t>(gridDim.x) * kWarps, lane);
  uint32_t magic = 0x4b000000u;
  asm volatile("" : "+r"(magic));  // (a register: the mask is the instruction's constant)
  while (run.more()) {
    // ---- up to 32 blocks of one pair ----
    const int n = run.count(), j = run.j;
    const int64_t pair = run.pair;
    const int tail = __ldg(kv.seq_lens + run.req) - j * B;  // tokens from the first of the blocks on
    int my_page = -1;
    if (lane < n) {
      my_page = __ldg(kv.page_table + pair * kv.max_blocks + j + lane);
      if (my_page < 0 || my_page >= kv.num_pages) {
        set_error(err, HS_EBIT_PAGE_RANGE);
        my_page = -1;
      }
    }
    // a place in the blocks that are there: block i (32: past them), row t
    struct Place {
      int i, t;
      unsigned left;  // blocks from i on
      __device__ __forceinline__ void block() { i = left ? __ffs(left) - 1 : 32; }
      __device__ __forceinline__ bool next(int valid) {  // true: the block ends
        t += kUnitRows;
        if (t < valid) return false;
        t = 0;
        left &= left - 1;
        block();
        return true;
      }
    };
    Place in{0, 0, __ballot_sync(0xffffffffu, my_page >= 0)};
    in.block();
    Place out = in;
    const auto valid_of = [&](int i) { return min(B, tail - i * B); };
    int unit_in = 0, unit_out = 0;
    const auto issue = [&]() {  // the next unit's rows, which lie together
      if (in.i < 32) {
        const int64_t row = static_cast<int64_t>(__shfl_sync(0xffffffffu, my_page, in.i)) * B + in.t;
        const int valid = valid_of(in.i), rows = min(valid - in.t, kUnitRows);
        const uint8_t* codes = static_cast<const uint8_t*>(kv.k_pages) + row * int4::row_bytes(D);
        const uint8_t* recs = reinterpret_cast<const uint8_t*>(kv.k_scales) + row * kRecord;
        const uint32_t to = mine_addr + unit_in * Unit<D>::kBytes;
#pragma unroll
        for (int x = 0; x < Unit<D>::kCodes; x += 512)
          if (x + lane * 16 < rows * int4::row_bytes(D)) copy16_async(to + x + lane * 16, codes + x + lane * 16);
        if (lane < rows) {
          if constexpr (kRecord == 16)
            copy16_async(to + Unit<D>::kCodes + lane * 16, recs + lane * 16);
          else
            copy8_async(to + Unit<D>::kCodes + lane * 8, recs + lane * 8);
        }
        in.next(valid);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      unit_in = unit_in + 1 == kUnits ? 0 : unit_in + 1;
    };
#pragma unroll
    for (int u = 0; u < kUnits - 1; ++u) issue();
    float mn[8], mx[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      mn[c] = INFINITY;
      mx[c] = -INFINITY;
    }
    while (out.i < 32) {
      __syncwarp();  // the unit about to be filled has been read by every lane
      issue();
      asm volatile("cp.async.wait_group %0;" ::"n"(kUnits - 1) : "memory");
      __syncwarp();
      const uint8_t* unit = mine + unit_out * Unit<D>::kBytes;
      unit_out = unit_out + 1 == kUnits ? 0 : unit_out + 1;
      const int valid = valid_of(out.i), rows = min(valid - out.t, kUnitRows);
      const uint8_t* codes = unit + d0 / 2;
      const uint16_t* recs = reinterpret_cast<const uint16_t*>(unit + Unit<D>::kCodes) + d0 / kQuantGroup;
      const auto two = [&](int r0, int r1) {  // the lane's channels of two rows
        float x[8], y[8];
        Codes8{*reinterpret_cast<const uint32_t*>(codes + r0 * int4::row_bytes(D)), recs[r0 * (kRecord / 2)],
               recs[r0 * (kRecord / 2) + D / kQuantGroup]}.get(x, magic);
        Codes8{*reinterpret_cast<const uint32_t*>(codes + r1 * int4::row_bytes(D)), recs[r1 * (kRecord / 2)],
               recs[r1 * (kRecord / 2) + D / kQuantGroup]}.get(y, magic);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          mn[c] = fminf(mn[c], fminf(x[c], y[c]));
          mx[c] = fmaxf(mx[c], fmaxf(x[c], y[c]));
        }
      };
      if (rows == kUnitRows) {
        codes += rs * int4::row_bytes(D);
        recs += rs * (kRecord / 2);
#pragma unroll
        for (int t = 0; t < kUnitRows; t += 2 * RPL) two(t, t + RPL);
      } else {
#pragma unroll 1
        for (int t = 0; t < rows; t += 2 * RPL) two(min(t + rs, rows - 1), min(t + RPL + rs, rows - 1));  // (a repeated row changes nothing)
      }
      const int now = out.i;
      if (!out.next(valid)) continue;
      // the row slots joined: a lane keeps half of its channels each time
      int at = d0;
#pragma unroll
      for (int off = LPR, w = 4; off < 32; off <<= 1, w >>= 1) {
        const bool upper = lane & off;
#pragma unroll
        for (int c = 0; c < w; ++c) {
          const float a = upper ? mn[c + w] : mn[c], b = upper ? mx[c + w] : mx[c];
          const float oa = __shfl_xor_sync(0xffffffffu, upper ? mn[c] : mn[c + w], off);
          const float ob = __shfl_xor_sync(0xffffffffu, upper ? mx[c] : mx[c + w], off);
          mn[c] = fminf(a, oa);
          mx[c] = fmaxf(b, ob);
        }
        at += upper ? w : 0;
      }
      constexpr int kKept = 8 / RPL;
      const int64_t o = (pair * kv.max_blocks + j + now) * D + at;
      __nv_bfloat162 lo[kKept / 2], hi[kKept / 2];
#pragma unroll
      for (int c = 0; c < kKept / 2; ++c) {  // outward: the stored box still contains every dequantised key
        lo[c].x = __float2bfloat16_rd(mn[2 * c]);
        lo[c].y = __float2bfloat16_rd(mn[2 * c + 1]);
        hi[c].x = __float2bfloat16_ru(mx[2 * c]);
        hi[c].y = __float2bfloat16_ru(mx[2 * c + 1]);
      }
      if constexpr (kKept == 4) {
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(smin) + o) = *reinterpret_cast<const uint2*>(lo);
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(smax) + o) = *reinterpret_cast<const uint2*>(hi);
      } else {
        *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(smin) + o) = *reinterpret_cast<const uint32_t*>(lo);
        *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(smax) + o) = *reinterpret_cast<const uint32_t*>(hi);
      }
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        mn[c] = INFINITY;
        mx[c] = -INFINITY;
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();
    run.on(n);
  }
}

template <int D>
cudaError_t launch_int4(const KvView& kv, int first_block, int nblocks, void* smin, void* smax, unsigned* err, int sms,
                        cudaStream_t st) {
  // a warp for each block at most
  const int64_t most = (static_cast<int64_t>(kv.batch) * kv.hkv * nblocks + kWarps - 1) / kWarps;
  const int resident = sms * 3;
  const unsigned grid = static_cast<unsigned>(most < resident ? most : resident);
  constexpr size_t smem = static_cast<size_t>(kWarps) * kUnits * Unit<D>::kBytes;
  static std::atomic<uint64_t> allowed{0};
  if (cudaError_t e = allow_dynamic_smem_once(allowed, summaries_int4_kernel<D>, smem); e != cudaSuccess) return e;
  return launch_pdl(summaries_int4_kernel<D>, dim3(grid), dim3(kWarps * 32), smem, st, kv, first_block, smin, smax, err);
}

template <int D>
cudaError_t launch_d(const KvView& kv, int first_block, int nblocks, void* smin, void* smax,
                     unsigned* err, int sms, cudaStream_t st) {
  switch (kv.kv_dtype) {
    case HS_KV_F32: return launch_k<D, HS_KV_F32>(kv, first_block, nblocks, smin, smax, err, sms, st);
    case HS_KV_BF16: return launch_k<D, HS_KV_BF16>(kv, first_block, nblocks, smin, smax, err, sms, st);
    case HS_KV_FP8E4M3_G32: return launch_k<D, HS_KV_FP8E4M3_G32>(kv, first_block, nblocks, smin, smax, err, sms, st);
    case HS_KV_INT4_G32: return launch_int4<D>(kv, first_block, nblocks, smin, smax, err, sms, st);
    default: return launch_block<D>(kv, first_block, nblocks, smin, smax, err, sms, st);
  }
}

}  // namespace

cudaError_t launch_summaries(const KvView& kv, int first_block, void* smin, void* smax,
                             unsigned* err, int sms, cudaStream_t st) {
  const int nblocks = kv.max_blocks - first_block;
  if (nblocks <= 0 || kv.batch == 0) return cudaSuccess;
  return kv.head_dim == 128 ? launch_d<128>(kv, first_block, nblocks, smin, smax, err, sms, st)
                            : launch_d<64>(kv, first_block, nblocks, smin, smax, err, sms, st);
}

}  // namespace hs
