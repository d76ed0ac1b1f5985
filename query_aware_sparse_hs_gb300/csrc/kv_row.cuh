// C channels of one row of the paged cache, of any kind, as fp32.
#pragma once

#include "int4.cuh"

namespace hs {

template <int C, int KIND>
__device__ __forceinline__ void load_row(const void* pages, const float* scales, int page, int64_t row,
                                         int D, int d0, float (&x)[C]) {
  if constexpr (KIND == HS_KV_F32) {
    const float* p = static_cast<const float*>(pages) + row * D + d0;
#pragma unroll
    for (int c = 0; c < C; ++c) x[c] = __ldg(p + c);
  } else if constexpr (KIND == HS_KV_BF16) {
    const uint16_t* p = static_cast<const uint16_t*>(pages) + row * D + d0;
#pragma unroll
    for (int c = 0; c < C; ++c) x[c] = bf16_bits_to_float(__ldg(reinterpret_cast<const unsigned short*>(p + c)));
  } else if constexpr (KIND == HS_KV_INT4_G32) {
    const uint8_t* p = static_cast<const uint8_t*>(pages) + row * int4::row_bytes(D) + d0 / 2;
    const float2 q = int4::load_scale(scales, row, D, d0 / kQuantGroup);
#pragma unroll
    for (int c = 0; c < C; c += 2) {
      const uint32_t two = __ldg(p + c / 2);
      x[c] = fmaf(q.x, static_cast<float>(static_cast<int>(two & 15u) - 8), q.y);
      x[c + 1] = fmaf(q.x, static_cast<float>(static_cast<int>(two >> 4) - 8), q.y);
    }
  } else {
    const uint8_t* p = static_cast<const uint8_t*>(pages) + row * D + d0;
    const float s = __ldg(KIND == HS_KV_FP8E4M3_BLOCK ? scales + page : scales + row * (D / kQuantGroup) + d0 / kQuantGroup);
#pragma unroll
    for (int c = 0; c < C; c += 2) {
      const uint16_t two = static_cast<uint16_t>(__ldg(p + c)) | (static_cast<uint16_t>(__ldg(p + c + 1)) << 8);
      float2 f = e4m3x2_to_float2(two);
      x[c] = f.x * s;
      x[c + 1] = f.y * s;
    }
  }
}

}  // namespace hs
