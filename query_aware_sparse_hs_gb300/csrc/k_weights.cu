// Attention weights accumulated per token ("KV 稀疏化" wiki §2, H2O: the tokens that
// attention has looked at most are kept): for every token t of the selected blocks
//   weights[b][kvh][t] += sum over the group's heads of e^(scale q.K[t] - lse),
// lse being what the step's attention left, so that every head adds 1 in all.
#include "hs_internal.h"
#include "kv_row.cuh"

namespace hs {
namespace {

constexpr int kWarps = 4;

// A warp takes a selected block, a token at a time; lane = D / 32 channels.
template <int C, int KIND>
__global__ __launch_bounds__(kWarps * 32) void weights_kernel(KvView kv, WeightsArgs a, unsigned* err) {
  constexpr int D = C * 32;
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * kWarps;
  const int64_t units = static_cast<int64_t>(kv.batch) * kv.hkv * a.capacity;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); u < units; u += warps) {
    const int64_t pair = u / a.capacity;
    const int i = static_cast<int>(u - pair * a.capacity);
    const int cnt = __ldg(a.sel_count + pair);
    if (cnt > a.capacity && i == 0 && lane == 0) set_error(err, HS_EBIT_CAPACITY);
    if (i >= cnt) continue;
    const int b = static_cast<int>(pair / kv.hkv), kvh = static_cast<int>(pair - static_cast<int64_t>(b) * kv.hkv);
    const int L = __ldg(kv.seq_lens + b), nb = min(ceil_div(max(L, 0), kv.block), kv.max_blocks);
    const int j = __ldg(a.sel + u);
    if (j < 0 || j >= nb) {
      if (lane == 0) set_error(err, HS_EBIT_BLOCK_RANGE);
      continue;
    }
    const int page = __ldg(kv.page_table + pair * kv.max_blocks + j);
    if (page < 0 || page >= kv.num_pages) {
      if (lane == 0) set_error(err, HS_EBIT_PAGE_RANGE);
      continue;
    }
    const int valid = min(kv.block, L - j * kv.block);
    float* out = a.weights + (pair * kv.max_blocks + j) * kv.block;
    for (int t = 0; t < valid; ++t) {
      float x[C];
      load_row<C, KIND>(kv.k_pages, kv.k_scales, page, static_cast<int64_t>(page) * kv.block + t, D, lane * C, x);
      float sum = 0.0f;
      for (int h = 0; h < kv.group; ++h) {
        const int64_t head = static_cast<int64_t>(b) * kv.hq + kvh * kv.group + h;
        float dot = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c)
          dot = fmaf(KIND == HS_KV_F32 ? static_cast<const float*>(a.q)[head * D + lane * C + c]
                                       : __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[head * D + lane * C + c]),
                     x[c], dot);
        const float lse = __ldg(a.lse + head);
        if (lse != -INFINITY) sum += expf(fmaf(warp_sum(dot), a.scale, -lse));
      }
      if (lane == 0) atomicAdd(out + t, sum);  // (a block may be selected twice: equal sums, in either order)
    }
  }
}

template <int C>
cudaError_t launch_c(const KvView& kv, const WeightsArgs& a, int sms, unsigned* err, cudaStream_t st) {
  const int64_t most = (static_cast<int64_t>(kv.batch) * kv.hkv * a.capacity + kWarps - 1) / kWarps;
  const dim3 grid(static_cast<unsigned>(most < sms * 16 ? most : sms * 16)), block(kWarps * 32);
  switch (kv.kv_dtype) {
    case HS_KV_F32: return launch_pdl(weights_kernel<C, HS_KV_F32>, grid, block, 0, st, kv, a, err);
    case HS_KV_BF16: return launch_pdl(weights_kernel<C, HS_KV_BF16>, grid, block, 0, st, kv, a, err);
    case HS_KV_FP8E4M3_G32: return launch_pdl(weights_kernel<C, HS_KV_FP8E4M3_G32>, grid, block, 0, st, kv, a, err);
    case HS_KV_INT4_G32: return launch_pdl(weights_kernel<C, HS_KV_INT4_G32>, grid, block, 0, st, kv, a, err);
    default: return launch_pdl(weights_kernel<C, HS_KV_FP8E4M3_BLOCK>, grid, block, 0, st, kv, a, err);
  }
}

}  // namespace

bool weights_fits(const KvView& kv, const WeightsArgs&) { return static_cast<int64_t>(kv.batch) * kv.hkv <= INT32_MAX; }

cudaError_t launch_weights(const KvView& kv, const WeightsArgs& a, int sms, unsigned* err, cudaStream_t st) {
  if (kv.batch == 0) return cudaSuccess;
  return kv.head_dim == 128 ? launch_c<4>(kv, a, sms, err, st) : launch_c<2>(kv, a, sms, err, st);
}

}  // namespace hs
