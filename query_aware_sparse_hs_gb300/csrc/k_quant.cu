// Grouped e4m3 quantisation of K/V rows ("分块稀疏注意力与KV Cache量化" §2.4:
// channels split into groups with one scale each; §3.2: group size 32).
// One warp per row; lane owns C = D/32 consecutive channels, so a 32-channel
// group spans 32/C lanes and its amax is a shuffle reduction inside them.
#include "hs_internal.h"
#include "int4.cuh"

namespace hs {
namespace {

constexpr int kWarps = 8;

template <int C, bool F32>
__global__ __launch_bounds__(kWarps * 32) void quant_kernel(const void* __restrict__ src, int64_t rows,
                                                           uint8_t* __restrict__ codes,
                                                           float* __restrict__ scales) {
  constexpr int D = C * 32;
  constexpr int kLanesPerGroup = kQuantGroup / C;
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (row >= rows) return;
  float x[C];
  if constexpr (F32) {
    const float* p = static_cast<const float*>(src) + row * D + lane * C;
#pragma unroll
    for (int c = 0; c < C; ++c) x[c] = p[c];
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(src) + row * D + lane * C;
#pragma unroll
    for (int c = 0; c < C; ++c) x[c] = bf16_bits_to_float(p[c]);
  }
  uint8_t out[C];
  const float scale = quantize_e4m3_lane<C>(x, out);
  uint8_t* q = codes + row * D + lane * C;
#pragma unroll
  for (int c = 0; c < C; ++c) q[c] = out[c];
  if ((lane % kLanesPerGroup) == 0) scales[row * (D / kQuantGroup) + lane / kLanesPerGroup] = scale;
}

template <int C>
cudaError_t launch_c(const void* src, bool f32, int64_t rows, uint8_t* codes, float* scales,
                     cudaStream_t st) {
  const int64_t grid = (rows + kWarps - 1) / kWarps;
  if (f32)
    quant_kernel<C, true><<<static_cast<unsigned>(grid), kWarps * 32, 0, st>>>(src, rows, codes, scales);
  else
    quant_kernel<C, false><<<static_cast<unsigned>(grid), kWarps * 32, 0, st>>>(src, rows, codes, scales);
  return cudaGetLastError();
}

// The 4-bit format (int4.cuh): a thread takes 8 neighbouring channels, so that a
// group is 4 threads and every access of a warp is one run of memory.  4 million rows of
// 128 bf16 values: read back in 230 us, 0.86 of the copy rate (four vectors to a thread
// 225, but 8192 rows 2.2 us for 1.8); quantised in 260 us, 0.76, bound by instructions
// (with values one at a time and a division by 7: 317).
constexpr int kThreads4 = 256;

constexpr int kFlight = 2;  // vectors of a thread, kThreads4 apart, both loaded before one is used

// Rows of 2^LOG vectors of 8 channels.
template <bool F32, int LOG>
__global__ __launch_bounds__(kThreads4) void quant_int4_kernel(const void* __restrict__ src, int64_t vectors,
                                                              uint8_t* __restrict__ codes, void* __restrict__ scales) {
  pdl_trigger();
  pdl_wait();
  const int64_t v0 = static_cast<int64_t>(blockIdx.x) * (kThreads4 * kFlight) + threadIdx.x;
  float4 raw[kFlight][F32 ? 2 : 1];
#pragma unroll
  for (int u = 0; u < kFlight; ++u) {
    const int64_t at = min(v0 + u * kThreads4, vectors - 1);  // (vectors is a multiple of 4: groups are whole)
    const float4* p = static_cast<const float4*>(src) + at * (F32 ? 2 : 1);
    raw[u][0] = __ldg(p);
    if constexpr (F32) raw[u][1] = __ldg(p + 1);
  }
#pragma unroll
  for (int u = 0; u < kFlight; ++u) {
    const int64_t v = v0 + u * kThreads4;
    const float4 a = raw[u][0];
    float x[8];
    if constexpr (F32) {
      const float4 b = raw[u][1];
      x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
      x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
      const uint32_t r[4] = {__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(a.z), __float_as_uint(a.w)};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(r[i] << 16);
        x[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
      }
    }
    int4::Range r = int4::range_of(x);
    r.join_lane(1);
    r.join_lane(2);
    if (v >= vectors) continue;
    const int4::Scale q = int4::scale_of(r);
    reinterpret_cast<uint32_t*>(codes)[v] = int4::encode8(x, q);
    if ((v & 3) == 0) int4::store_scale(scales, v >> LOG, 8 << LOG, static_cast<int>(v & ((1 << LOG) - 1)) / 4, q);
  }
}

template <bool F32, int LOG>
__global__ __launch_bounds__(kThreads4) void dequant_int4_kernel(const uint8_t* __restrict__ codes, const void* __restrict__ scales,
                                                                int64_t vectors, void* __restrict__ dst) {
  pdl_trigger();
  pdl_wait();
  const int64_t v0 = static_cast<int64_t>(blockIdx.x) * (kThreads4 * kFlight) + threadIdx.x;
  uint32_t w[kFlight];
  float2 q[kFlight];
#pragma unroll
  for (int u = 0; u < kFlight; ++u) {
    const int64_t at = min(v0 + u * kThreads4, vectors - 1);
    w[u] = __ldg(reinterpret_cast<const uint32_t*>(codes) + at);
    q[u] = int4::load_scale(scales, at >> LOG, 8 << LOG, static_cast<int>(at & ((1 << LOG) - 1)) / 4);
  }
#pragma unroll
  for (int u = 0; u < kFlight; ++u) {
    const int64_t v = v0 + u * kThreads4;
    if (v >= vectors) return;
    float x[8];
    int4::decode8(w[u], q[u].x, q[u].y, x);
    if constexpr (F32) {
      float4* p = static_cast<float4*>(dst) + 2 * v;
      p[0] = make_float4(x[0], x[1], x[2], x[3]);
      p[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
      __nv_bfloat162 y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      static_cast<uint4*>(dst)[v] = *reinterpret_cast<const uint4*>(y);
    }
  }
}

template <int LOG>
cudaError_t launch_quant4(const void* src, bool f32, int64_t vectors, uint8_t* codes, void* scales, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>((vectors + kThreads4 * kFlight - 1) / (kThreads4 * kFlight)));
  return f32 ? launch_pdl(quant_int4_kernel<true, LOG>, grid, dim3(kThreads4), 0, st, src, vectors, codes, scales)
             : launch_pdl(quant_int4_kernel<false, LOG>, grid, dim3(kThreads4), 0, st, src, vectors, codes, scales);
}
template <int LOG>
cudaError_t launch_dequant4(const uint8_t* codes, const void* scales, int64_t vectors, void* dst, bool f32, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>((vectors + kThreads4 * kFlight - 1) / (kThreads4 * kFlight)));
  return f32 ? launch_pdl(dequant_int4_kernel<true, LOG>, grid, dim3(kThreads4), 0, st, codes, scales, vectors, dst)
             : launch_pdl(dequant_int4_kernel<false, LOG>, grid, dim3(kThreads4), 0, st, codes, scales, vectors, dst);
}

}  // namespace

cudaError_t launch_quantize_int4(const void* src, bool src_f32, int64_t rows, int head_dim, uint8_t* codes, void* scales,
                                 cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  const int64_t vectors = rows * (head_dim / 8);
  switch (head_dim) {
    case 64: return launch_quant4<3>(src, src_f32, vectors, codes, scales, st);
    case 128: return launch_quant4<4>(src, src_f32, vectors, codes, scales, st);
    default: return launch_quant4<5>(src, src_f32, vectors, codes, scales, st);
  }
}

cudaError_t launch_dequantize_int4(const uint8_t* codes, const void* scales, int64_t rows, int head_dim, void* dst, bool dst_f32,
                                   cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  const int64_t vectors = rows * (head_dim / 8);
  switch (head_dim) {
    case 64: return launch_dequant4<3>(codes, scales, vectors, dst, dst_f32, st);
    case 128: return launch_dequant4<4>(codes, scales, vectors, dst, dst_f32, st);
    default: return launch_dequant4<5>(codes, scales, vectors, dst, dst_f32, st);
  }
}

cudaError_t launch_quantize(const void* src, bool src_f32, int64_t rows, int head_dim,
                            uint8_t* codes, float* scales, cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  switch (head_dim) {
    case 64: return launch_c<2>(src, src_f32, rows, codes, scales, st);
    case 128: return launch_c<4>(src, src_f32, rows, codes, scales, st);
    case 256: return launch_c<8>(src, src_f32, rows, codes, scales, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace hs
