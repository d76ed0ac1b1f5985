// Eviction of the tokens that attention has looked at least ("KV 稀疏化" wiki §2, H2O:
// heavy hitters by accumulated weight, the sink and the recent tokens kept): of every
// (request, kv head) the first sink and the last recent tokens and the heaviest of the
// others, budget tokens in all, are gathered in order into the pages of another cache.
//   evict_select_kernel  which tokens: the weight of the last that stays by a radix
//                        search, then their indices in ascending order (kept)
//   evict_gather_kernel  their rows, scales and weights to the new pages
#include "hs_internal.h"

namespace hs {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 256;

__device__ __forceinline__ uint32_t weight_key(float w) {  // NaN last, -0 as 0
  if (isnan(w)) return 0u;
  const uint32_t u = w == 0.0f ? 0u : __float_as_uint(w);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// CTA = (request, kv head).
__global__ __launch_bounds__(kSelThreads) void evict_select_kernel(KvView kv, EvictArgs a, unsigned* err) {
  __shared__ uint32_t s_hist[kBins];
  __shared__ uint32_t s_found[2];  // digit, keys above it
  __shared__ int s_above[kSelWarps], s_same[kSelWarps];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t pair = blockIdx.x;
  const int b = static_cast<int>(pair / kv.hkv);
  const int64_t most = static_cast<int64_t>(kv.max_blocks) * kv.block;
  int L = max(__ldg(kv.seq_lens + b), 0);
  if (L > most) {
    if (tid == 0) set_error(err, HS_EBIT_BLOCK_RANGE);
    L = static_cast<int>(most);
  }
  int32_t* kept = a.kept + pair * a.budget;
  if (L <= a.budget) {
    for (int i = tid; i < a.budget; i += kSelThreads) kept[i] = i < L ? i : -1;
    return;
  }
  const float* w = a.weights + pair * most;
  const int first = a.sink, last = L - a.recent;  // the tokens that are chosen from
  const int need = a.budget - a.sink - a.recent;
  for (int i = tid; i < a.sink; i += kSelThreads) kept[i] = i;
  for (int i = tid; i < a.recent; i += kSelThreads) kept[a.budget - a.recent + i] = last + i;
  if (need == 0) return;
  // ---- the key of the last that stays, and how many of the same key do ----
  uint32_t prefix = 0u, mask = 0u;
  int rank = need;  // among the keys that share the prefix
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < kBins; i += kSelThreads) s_hist[i] = 0u;
    __syncthreads();
    for (int t = first + tid; t < last; t += kSelThreads) {
      const uint32_t k = weight_key(__ldg(w + t));
      if ((k & mask) == prefix) atomicAdd(&s_hist[(k >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (tid == 0) {
      uint32_t above = 0u;
      int d = 255;
      while (d > 0 && above + s_hist[d] < static_cast<uint32_t>(rank)) above += s_hist[d--];
      s_found[0] = d;
      s_found[1] = above;
    }
    __syncthreads();
    prefix |= s_found[0] << shift;
    mask |= 255u << shift;
    rank -= static_cast<int>(s_found[1]);
  }
  // ---- their indices: a warp takes a run of the tokens ----
  const int run = ((last - first + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
  const int t0 = min(last, first + warp * run), t1 = min(last, t0 + run);
  int above = 0, same = 0;
  for (int t = t0 + lane; t < t1; t += 32) {
    const uint32_t k = weight_key(__ldg(w + t));
    above += k > prefix;
    same += k == prefix;
  }
  above = __reduce_add_sync(0xffffffffu, above);
  same = __reduce_add_sync(0xffffffffu, same);
  if (lane == 0) {
    s_above[warp] = above;
    s_same[warp] = same;
  }
  __syncthreads();
  above = same = 0;
  for (int i = 0; i < warp; ++i) {
    above += s_above[i];
    same += s_same[i];
  }
  for (int t = t0; t < t1; t += 32) {
    const uint32_t k = t + lane < t1 ? weight_key(__ldg(w + t + lane)) : 0u;
    const bool is_above = t + lane < t1 && k > prefix, is_same = t + lane < t1 && k == prefix;
    const unsigned ma = __ballot_sync(0xffffffffu, is_above), ms = __ballot_sync(0xffffffffu, is_same);
    const unsigned lower = (1u << lane) - 1u;
    const int same_here = same + __popc(ms & lower), above_here = above + __popc(ma & lower);
    // of the equal ones the first `rank` stay
    if (is_above || (is_same && same_here < rank)) kept[a.sink + above_here + min(same_here, rank)] = t + lane;
    above += __popc(ma);
    same += __popc(ms);
  }
}

constexpr int kRows = 32;  // rows of a CTA
constexpr int kGatherThreads = 128;

// CTA = kRows places of a (request, kv head)'s new pages.  row_bytes, scale_bytes: of a
// row of K (or V).
__global__ __launch_bounds__(kGatherThreads) void evict_gather_kernel(KvView kv, KvView dst, EvictArgs a, int chunks, int row_bytes,
                                                                      int scale_bytes, unsigned* err) {
  __shared__ int64_t s_from[kRows], s_to[kRows];  // rows of the pools, -1: none
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x;
  const int64_t pair = blockIdx.x / chunks;
  const int i0 = static_cast<int>(blockIdx.x - pair * chunks) * kRows, B = kv.block;
  const int b = static_cast<int>(pair / kv.hkv);
  if (i0 == 0 && tid == 0 && pair == static_cast<int64_t>(b) * kv.hkv) {
    // (the only reader of lengths here, so that they may be written in place)
    const int64_t most = static_cast<int64_t>(kv.max_blocks) * B;
    const int64_t L = min(static_cast<int64_t>(max(kv.seq_lens[b], 0)), most);
    const_cast<int32_t*>(dst.seq_lens)[b] = static_cast<int>(min(L, static_cast<int64_t>(a.budget)));
  }
  if (tid < kRows) {
    const int i = i0 + tid;
    const int t = i < a.budget ? a.kept[pair * a.budget + i] : -1;
    int64_t from = -1, to = -1;
    if (t >= 0) {
      const int p = __ldg(kv.page_table + pair * kv.max_blocks + t / B);
      const int q = __ldg(dst.page_table + pair * dst.max_blocks + i / B);
      if (p < 0 || p >= kv.num_pages || q < 0 || q >= dst.num_pages) {
        set_error(err, HS_EBIT_PAGE_RANGE);
      } else {
        from = static_cast<int64_t>(p) * B + t % B;
        to = static_cast<int64_t>(q) * B + i % B;
        if (a.dst_weights) a.dst_weights[pair * dst.max_blocks * B + i] = __ldg(a.weights + pair * kv.max_blocks * B + t);
      }
    }
    s_from[tid] = from;
    s_to[tid] = to;
  }
  __syncthreads();
  const int pieces = row_bytes / 16, each = pieces * 2;
  for (int n = tid; n < kRows * each; n += kGatherThreads) {
    const int r = n / each, x = n - r * each;
    const bool v = x >= pieces;
    const int at = (v ? x - pieces : x) * 16;
    if (s_from[r] < 0) continue;
    const char* src = static_cast<const char*>(v ? kv.v_pages : kv.k_pages) + s_from[r] * row_bytes + at;
    char* to = static_cast<char*>(const_cast<void*>(v ? dst.v_pages : dst.k_pages)) + s_to[r] * row_bytes + at;
    *reinterpret_cast<uint4*>(to) = __ldg(reinterpret_cast<const uint4*>(src));
  }
  const int words = scale_bytes / 4;
  for (int n = tid; n < kRows * words * 2; n += kGatherThreads) {
    const int r = n / (words * 2), x = n - r * words * 2;
    const bool v = x >= words;
    const int at = v ? x - words : x;
    if (s_from[r] < 0) continue;
    const uint32_t* src = reinterpret_cast<const uint32_t*>(v ? kv.v_scales : kv.k_scales) + s_from[r] * words + at;
    uint32_t* to = reinterpret_cast<uint32_t*>(const_cast<float*>(v ? dst.v_scales : dst.k_scales)) + s_to[r] * words + at;
    *to = __ldg(src);
  }
}

}  // namespace

int64_t evict_ctas(const KvView& kv, int budget) {
  return static_cast<int64_t>(kv.batch) * kv.hkv * ceil_div(budget, kRows);
}

cudaError_t launch_evict(const KvView& kv, const KvView& dst, const EvictArgs& a, unsigned* err, cudaStream_t st) {
  if (kv.batch == 0) return cudaSuccess;
  cudaError_t e = launch_pdl(evict_select_kernel, dim3(kv.batch * kv.hkv), dim3(kSelThreads), 0, st, kv, a, err);
  if (e != cudaSuccess) return e;
  const int elem2 = kv.kv_dtype == HS_KV_F32 ? 8 : kv.kv_dtype == HS_KV_BF16 ? 4 : kv.kv_dtype == HS_KV_INT4_G32 ? 1 : 2;
  const int scale_bytes = kv.kv_dtype >= HS_KV_FP8E4M3_G32 ? kv.head_dim / kQuantGroup * 4 : 0;
  return launch_pdl(evict_gather_kernel, dim3(static_cast<unsigned>(evict_ctas(kv, a.budget))), dim3(kGatherThreads), 0, st, kv, dst, a,
                    ceil_div(a.budget, kRows), kv.head_dim * elem2 / 2, scale_bytes, err);
}

}  // namespace hs
