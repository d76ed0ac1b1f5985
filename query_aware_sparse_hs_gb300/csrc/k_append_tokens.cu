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
// One launch.  A CTA takes one (touched block, kv head, K or V): it owns the
// page and its scale, so nothing is exchanged between CTAs and there are no
// atomics.  The other CTAs rotate Q, one warp per row and 16 heads, so that the
// row's cos and sin are read once for 16 heads.  A thread holds 16 channels of a
// row as two vectors of 8 chosen so that both members of every rotated pair are
// its own.  Memory-bound (prompts) or latency-bound (single tokens).
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
__device__ __forceinline__ int last_not_above(int n, int64_t x, int lane, F key) {
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

template <bool F32>
__device__ __forceinline__ void load8(const void* p, int64_t at, float (&x)[8]) {
  if constexpr (F32) {
    const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
    const float4 u = __ldg(s), w = __ldg(s + 1);
    x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
    x[4] = w.x; x[5] = w.y; x[6] = w.z; x[7] = w.w;
  } else {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at));
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
__device__ __forceinline__ void rotate(float (&a)[8], float (&b)[8], const Angles& t, bool interleaved) {
  if (interleaved) {
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

template <int D, bool F32>
__device__ void rotate_q(const KvView& kv, const AppendTokensArgs& a, int64_t unit, int lane, unsigned* err) {
  constexpr int TPR = D / 16, HPP = 32 / TPR;  // threads per head, heads per step
  const int chunks = ceil_div(kv.hq, kQHeads);
  const int64_t row = unit / chunks;
  if (row >= a.rows) return;
  const int h0 = static_cast<int>(unit - row * chunks) * kQHeads;
  int b = static_cast<int>(row);
  int64_t behind = 1;  // tokens from this row's to the end of its request
  if (a.offsets) {
    b = last_not_above(kv.batch, row, lane, [&](int i) { return static_cast<int64_t>(__ldg(a.offsets + i)); });
    const int64_t o0 = a.offsets[b], o1 = a.offsets[b + 1];
    if (row < o0 || row >= o1 || o1 > a.rows) return;  // behind the last request, or offsets reported by the K and V units
    if (o1 - o0 > kv.seq_lens[b]) return;
    behind = o1 - row;
  }
  const int64_t p = static_cast<int64_t>(kv.seq_lens[b]) - behind;
  if (p < 0) return;
  const int64_t pos = a.positions ? a.positions[row] : p;
  if (a.rotary > 0 && (pos < 0 || pos >= a.table_rows)) {
    if (lane == 0) set_error(err, HS_EBIT_POSITION);
    return;
  }
  const int s = lane % TPR;
  const Slot t = slot_of(s, a.rotary, a.interleaved);
  Angles ang;
  if (t.rotated) load_angles(a.cos_sin, a.rotary, pos, s, ang);
  const int64_t in = row * a.q_stride, out = row * a.q_out_stride;
#pragma unroll
  for (int i = 0; i < kQHeads / HPP; ++i) {
    const int h = h0 + i * HPP + lane / TPR;
    if (h < kv.hq) {
      float x[8], y[8];
      load8<F32>(a.q, in + h * D + t.ca, x);
      load8<F32>(a.q, in + h * D + t.cb, y);
      if (t.rotated) rotate(x, y, ang, a.interleaved);
      store8<F32>(a.q_out, out + h * D + t.ca, x);
      store8<F32>(a.q_out, out + h * D + t.cb, y);
    }
  }
}

template <int D, int KIND>
__global__ __launch_bounds__(kThreads) void append_tokens_kernel(KvView kv, AppendTokensArgs a, int64_t kv_units,
                                                                 unsigned* err) {
  constexpr bool F32 = KIND == HS_KV_F32;
  constexpr int TPR = D / 16, RPP = kThreads / TPR;  // threads per row, rows per pass
  __shared__ float s_mn[kWarps][D], s_mx[kWarps][D];
  __shared__ float s_amax[kWarps];
  __shared__ int s_any[kWarps];
  __shared__ unsigned s_group[RPP][D / kQuantGroup];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (static_cast<int64_t>(blockIdx.x) >= kv_units) {
    rotate_q<D, F32>(kv, a, (blockIdx.x - kv_units) * kWarps + warp, lane, err);
    return;
  }
  // ---- which block ----
  const bool is_k = (blockIdx.x & 1) == 0;
  const int64_t rest = blockIdx.x >> 1;
  const int64_t slot = rest / kv.hkv;
  const int kvh = static_cast<int>(rest - slot * kv.hkv);
  const int B = kv.block;
  int b = static_cast<int>(slot);
  int64_t o0 = slot;
  int n = 1, x = 0;
  if (a.offsets) {
    // request b has the slots from offsets[b] / B + 2 b on: enough for every
    // block its rows can touch, wherever in a block they begin
    b = last_not_above(kv.batch, slot, lane, [&](int i) { return static_cast<int64_t>(__ldg(a.offsets + i)) / B + 2 * i; });
    o0 = a.offsets[b];
    const int64_t o1 = a.offsets[b + 1];
    if (o0 < 0 || o1 < o0 || o1 > a.rows) {
      if (tid == 0) set_error(err, HS_EBIT_BLOCK_RANGE);
      return;
    }
    n = static_cast<int>(o1 - o0);
    x = static_cast<int>(slot - (o0 / B + 2 * static_cast<int64_t>(b)));
    if (x < 0) return;
  }
  const int L = kv.seq_lens[b];
  if (n <= 0 || L <= 0) return;
  if (n > L) {
    if (tid == 0) set_error(err, HS_EBIT_BLOCK_RANGE);
    return;
  }
  const int first = L - n;  // cache position of the request's first new row
  const int64_t j64 = static_cast<int64_t>(first / B) + x;
  if (j64 > (L - 1) / B) return;
  const int j = static_cast<int>(j64);
  const int64_t pair = static_cast<int64_t>(b) * kv.hkv + kvh;
  if (j >= kv.max_blocks) {
    if (tid == 0) set_error(err, HS_EBIT_BLOCK_RANGE);
    return;
  }
  const int page = kv.page_table[pair * kv.max_blocks + j];
  if (page < 0 || page >= kv.num_pages) {
    if (tid == 0) set_error(err, HS_EBIT_PAGE_RANGE);
    return;
  }
  const int ra = max(0, first - j * B), rb = min(B, L - j * B);  // rows of the page that are new
  const void* src = is_k ? a.k : a.v;
  const int64_t stride = is_k ? a.k_stride : a.v_stride;
  const int64_t src0 = o0 + (static_cast<int64_t>(j) * B - first);  // + page row = source row
  void* pages = const_cast<void*>(is_k ? kv.k_pages : kv.v_pages);
  float* scales = const_cast<float*>(is_k ? kv.k_scales : kv.v_scales);
  const int64_t row0 = static_cast<int64_t>(page) * B;
  const int rotary = is_k ? a.rotary : 0;
  const bool box = is_k && a.smin != nullptr;
  const int s = tid % TPR, rs = tid / TPR;
  const Slot t = slot_of(s, rotary, a.interleaved);

  // the rotated channels of page row r; false where the position has no table row
  auto fetch = [&](int r, float (&u)[8], float (&w)[8]) {
    const int64_t sr = src0 + r;
    if (rotary > 0) {
      const int64_t pos = a.positions ? a.positions[sr] : static_cast<int64_t>(j) * B + r;
      if (pos < 0 || pos >= a.table_rows) {
        set_error(err, HS_EBIT_POSITION);
        return false;
      }
      load8<F32>(src, sr * stride + kvh * D + t.ca, u);
      load8<F32>(src, sr * stride + kvh * D + t.cb, w);
      if (t.rotated) {
        Angles ang;
        load_angles(a.cos_sin, rotary, pos, s, ang);
        rotate(u, w, ang, a.interleaved);
      }
    } else {
      load8<F32>(src, sr * stride + kvh * D + t.ca, u);
      load8<F32>(src, sr * stride + kvh * D + t.cb, w);
    }
    return true;
  };

  float mn[16], mx[16];
#pragma unroll
  for (int c = 0; c < 16; ++c) {
    mn[c] = INFINITY;
    mx[c] = -INFINITY;
  }
  auto widen = [&](const float (&u)[8], const float (&w)[8]) {
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      mn[c] = fminf(mn[c], u[c]);
      mx[c] = fmaxf(mx[c], u[c]);
      mn[8 + c] = fminf(mn[8 + c], w[c]);
      mx[8 + c] = fmaxf(mx[8 + c], w[c]);
    }
  };
  bool any = false;
  float amax = 0.0f;
  const int passes = ceil_div(rb - ra, RPP);
  for (int i = 0; i < passes; ++i) {
    const int r = ra + i * RPP + rs;
    float u[8], w[8];
    const bool live = r < rb && fetch(r, u, w);
    any |= live;
    if constexpr (KIND == HS_KV_FP8E4M3_G32) {
      // the row's threads are neighbours in one warp
      if (s < D / kQuantGroup) s_group[rs][s] = 0u;
      __syncwarp();
      if (live) {
        float p = 0.0f, q = 0.0f;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          p = fmaxf(p, fabsf(u[c]));
          q = fmaxf(q, fabsf(w[c]));
        }
        atomicMax(&s_group[rs][t.ca / kQuantGroup], __float_as_uint(p));
        atomicMax(&s_group[rs][t.cb / kQuantGroup], __float_as_uint(q));
      }
      __syncwarp();
      if (live) {
        const float ga = __uint_as_float(s_group[rs][t.ca / kQuantGroup]);
        const float gb = __uint_as_float(s_group[rs][t.cb / kQuantGroup]);
        const float sa = ga > 0.0f ? ga / 448.0f : 1.0f, sb = gb > 0.0f ? gb / 448.0f : 1.0f;
#pragma unroll
        for (int c = 0; c < 8; ++c) {  // IEEE division, as the quantiser of whole rows does
          u[c] = u[c] / sa;
          w[c] = w[c] / sb;
        }
        uint8_t* dst = static_cast<uint8_t*>(pages) + (row0 + r) * D;
        const uint2 cu = encode8(u, 1.0f), cw = encode8(w, 1.0f);
        *reinterpret_cast<uint2*>(dst + t.ca) = cu;
        *reinterpret_cast<uint2*>(dst + t.cb) = cw;
        if (s < D / kQuantGroup) {
          const float g = __uint_as_float(s_group[rs][s]);
          scales[(row0 + r) * (D / kQuantGroup) + s] = g > 0.0f ? g / 448.0f : 1.0f;
        }
        if (box) {
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            u[c] = decode1((c < 4 ? cu.x : cu.y) >> (8 * (c & 3)) & 0xffu) * sa;
            w[c] = decode1((c < 4 ? cw.x : cw.y) >> (8 * (c & 3)) & 0xffu) * sb;
          }
          widen(u, w);
        }
      }
      __syncwarp();
    } else if (live) {
      if constexpr (KIND == HS_KV_FP8E4M3_BLOCK) {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float p = fabsf(u[c]), q = fabsf(w[c]);
          amax = fmaxf(amax, p <= FLT_MAX ? p : 0.0f);
          amax = fmaxf(amax, q <= FLT_MAX ? q : 0.0f);
        }
      } else {
        store8<F32>(pages, (row0 + r) * D + t.ca, u);
        store8<F32>(pages, (row0 + r) * D + t.cb, w);
        if constexpr (KIND == HS_KV_BF16) {
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            u[c] = __bfloat162float(__float2bfloat16_rn(u[c]));
            w[c] = __bfloat162float(__float2bfloat16_rn(w[c]));
          }
        }
      }
      if (box) widen(u, w);
    }
  }

  float scale = 1.0f, inv = 1.0f;
  bool grown = false;
  if constexpr (KIND == HS_KV_FP8E4M3_BLOCK) {
    const float held = ra > 0 ? scales[page] : 0.0f;  // read by every thread before one of them writes it
    amax = warp_max(amax);
    if (lane == 0) s_amax[warp] = amax;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWarps; ++i) amax = fmaxf(amax, s_amax[i]);
    scale = block_scale(amax);
    if (ra > 0) {
      grown = !(held >= scale);  // (a scale that is not a number is replaced)
      if (!grown) scale = held;
    }
    inv = 1.0f / scale;
    if (grown) {
      // the rows already there, at the new scale
      const float f = held > 0.0f ? held * inv : 0.0f;
      for (int r = rs; r < ra; r += RPP) {
        uint4* p = reinterpret_cast<uint4*>(static_cast<uint8_t*>(pages) + (row0 + r) * D + 16 * s);
        const uint4 old = *p;
        const uint32_t in[4] = {old.x, old.y, old.z, old.w};
        uint32_t out[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float2 lo = e4m3x2_to_float2(static_cast<uint16_t>(in[c])), hi = e4m3x2_to_float2(static_cast<uint16_t>(in[c] >> 16));
          out[c] = __nv_cvt_float2_to_fp8x2(make_float2(lo.x * f, lo.y * f), __NV_SATFINITE, __NV_E4M3) |
                   static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(hi.x * f, hi.y * f), __NV_SATFINITE, __NV_E4M3)) << 16;
        }
        *p = make_uint4(out[0], out[1], out[2], out[3]);
      }
    }
    if (tid == 0 && (ra == 0 || grown)) scales[page] = scale;
    for (int i = 0; i < passes; ++i) {  // the rows again (from the caches), as codes
      const int r = ra + i * RPP + rs;
      float u[8], w[8];
      if (r < rb && fetch(r, u, w)) {
        uint8_t* dst = static_cast<uint8_t*>(pages) + (row0 + r) * D;
        *reinterpret_cast<uint2*>(dst + t.ca) = encode8(u, inv);
        *reinterpret_cast<uint2*>(dst + t.cb) = encode8(w, inv);
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
  __syncthreads();  // (also: the page's rows are written)
  int rows_written = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) rows_written |= s_any[i];
  if (!rows_written) return;  // every row's position was out of range
  const int d = tid;
  if (d >= D) return;
  float lo = s_mn[0][d], hi = s_mx[0][d];
#pragma unroll
  for (int i = 1; i < kWarps; ++i) {
    lo = fminf(lo, s_mn[i][d]);
    hi = fmaxf(hi, s_mx[i][d]);
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

template <int D>
cudaError_t launch_d(const KvView& kv, const AppendTokensArgs& a, int64_t kv_units, unsigned grid, unsigned* err,
                     cudaStream_t st) {
  const dim3 g(grid), t(kThreads);
  switch (kv.kv_dtype) {
    case HS_KV_F32: return launch_pdl(append_tokens_kernel<D, HS_KV_F32>, g, t, 0, st, kv, a, kv_units, err);
    case HS_KV_BF16: return launch_pdl(append_tokens_kernel<D, HS_KV_BF16>, g, t, 0, st, kv, a, kv_units, err);
    case HS_KV_FP8E4M3_G32: return launch_pdl(append_tokens_kernel<D, HS_KV_FP8E4M3_G32>, g, t, 0, st, kv, a, kv_units, err);
    default: return launch_pdl(append_tokens_kernel<D, HS_KV_FP8E4M3_BLOCK>, g, t, 0, st, kv, a, kv_units, err);
  }
}

// CTAs for the touched blocks: with offsets, request b's blocks have the slots
// from offsets[b] / B + 2 b on.
int64_t append_units(const KvView& kv, const AppendTokensArgs& a) {
  const int64_t slots = a.offsets ? a.rows / kv.block + 2 * static_cast<int64_t>(kv.batch) : kv.batch;
  return slots * kv.hkv * 2;
}
int64_t append_q_ctas(const KvView& kv, const AppendTokensArgs& a) {
  return a.q ? (a.rows * ceil_div(kv.hq, kQHeads) + kWarps - 1) / kWarps : 0;
}

}  // namespace

bool append_tokens_fits(const KvView& kv, const AppendTokensArgs& a) {
  return append_units(kv, a) + append_q_ctas(kv, a) <= INT32_MAX;
}

cudaError_t launch_append_tokens(const KvView& kv, const AppendTokensArgs& a, unsigned* err, cudaStream_t st) {
  const int64_t units = append_units(kv, a), ctas = units + append_q_ctas(kv, a);
  if (kv.batch == 0 || a.rows == 0) return cudaSuccess;
  return kv.head_dim == 128 ? launch_d<128>(kv, a, units, static_cast<unsigned>(ctas), err, st)
                            : launch_d<64>(kv, a, units, static_cast<unsigned>(ctas), err, st);
}

}  // namespace hs
