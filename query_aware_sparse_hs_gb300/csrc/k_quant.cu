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
// group is 4 threads and every access of a warp is one run of memory.
constexpr int kThreads4 = 256;

template <bool F32>
__global__ __launch_bounds__(kThreads4) void quant_int4_kernel(const void* __restrict__ src, int64_t vectors, int head_dim,
                                                              uint8_t* __restrict__ codes, void* __restrict__ scales) {
  pdl_trigger();
  pdl_wait();
  const int64_t v = static_cast<int64_t>(blockIdx.x) * kThreads4 + threadIdx.x;
  const int64_t at = min(v, vectors - 1);  // (vectors is a multiple of 4: groups are whole)
  float x[8];
  if constexpr (F32) {
    const float4* p = static_cast<const float4*>(src) + 2 * at;
    const float4 a = __ldg(p), b = __ldg(p + 1);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
    const uint4 a = __ldg(static_cast<const uint4*>(src) + at);
    const uint32_t r[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(r[i] << 16);
      x[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
    }
  }
  int4::Range r;
  r.clear();
#pragma unroll
  for (int i = 0; i < 8; ++i) r.add(x[i]);
  r.join_lane(1);
  r.join_lane(2);
  if (v >= vectors) return;
  const int4::Scale q = int4::scale_of(r);
  reinterpret_cast<uint32_t*>(codes)[v] = int4::encode8(x, q);
  if ((v & 3) == 0) {
    const int64_t row = v / (head_dim / 8);
    int4::store_scale(scales, row, head_dim, static_cast<int>(v - row * (head_dim / 8)) / 4, q);
  }
}

template <bool F32>
__global__ __launch_bounds__(kThreads4) void dequant_int4_kernel(const uint8_t* __restrict__ codes, const void* __restrict__ scales,
                                                                int64_t vectors, int head_dim, void* __restrict__ dst) {
  pdl_trigger();
  pdl_wait();
  const int64_t v = static_cast<int64_t>(blockIdx.x) * kThreads4 + threadIdx.x;
  if (v >= vectors) return;
  const int64_t row = v / (head_dim / 8);
  const float2 q = int4::load_scale(scales, row, head_dim, static_cast<int>(v - row * (head_dim / 8)) / 4);
  float x[8];
  int4::decode8(__ldg(reinterpret_cast<const uint32_t*>(codes) + v), q.x, q.y, x);
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

}  // namespace

cudaError_t launch_quantize_int4(const void* src, bool src_f32, int64_t rows, int head_dim, uint8_t* codes, void* scales,
                                 cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  const int64_t vectors = rows * (head_dim / 8);
  const dim3 grid(static_cast<unsigned>((vectors + kThreads4 - 1) / kThreads4));
  return src_f32 ? launch_pdl(quant_int4_kernel<true>, grid, dim3(kThreads4), 0, st, src, vectors, head_dim, codes, scales)
                 : launch_pdl(quant_int4_kernel<false>, grid, dim3(kThreads4), 0, st, src, vectors, head_dim, codes, scales);
}

cudaError_t launch_dequantize_int4(const uint8_t* codes, const void* scales, int64_t rows, int head_dim, void* dst, bool dst_f32,
                                   cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  const int64_t vectors = rows * (head_dim / 8);
  const dim3 grid(static_cast<unsigned>((vectors + kThreads4 - 1) / kThreads4));
  return dst_f32 ? launch_pdl(dequant_int4_kernel<true>, grid, dim3(kThreads4), 0, st, codes, scales, vectors, head_dim, dst)
                 : launch_pdl(dequant_int4_kernel<false>, grid, dim3(kThreads4), 0, st, codes, scales, vectors, head_dim, dst);
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
