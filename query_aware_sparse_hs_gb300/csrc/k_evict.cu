// Eviction of the tokens that attention has looked at least ("KV 稀疏化" wiki §2, H2O:
// heavy hitters by accumulated weight, the sink and the recent tokens kept): of every
// (request, kv head) the first sink and the last recent tokens and the heaviest of the
// others, budget tokens in all, are gathered in order into the pages of another cache.
//   evict_select_kernel  which tokens: the weight of the last that stays by a radix
//                        search, then their indices in ascending order (kept)
//   evict_gather_kernel  their rows, scales and weights to the new pages
#include <cooperative_groups.h>

#include "hs_internal.h"

namespace cg = cooperative_groups;

namespace hs {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kHeld = 16;             // keys of a thread that stay in registers
constexpr int kMostCtas = 8;          // of a cluster
constexpr int kBins = 2048;           // 11 bits of a key: 11, 11 and 10 are all of it

__device__ __forceinline__ uint32_t weight_key(float w) {  // NaN last, -0 as 0
  if (isnan(w)) return 0u;
  const uint32_t u = w == 0.0f ? 0u : __float_as_uint(w);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Cluster = (request, kv head).  The tokens that are chosen from are cut into a run for
// each warp of the cluster's CTAs, whose keys stay in registers, 16 to a thread (more are
// read again from the caches).  The key of the last token that stays is found from
// histograms of 11 bits at a time, which every CTA sums over the cluster through
// distributed shared memory; a bin that is taken whole ends the search.
// Latency-bound, by two loads that follow one another, the barriers of the cluster (0.6 us
// each) and what lies between them: with a budget of 64, so that little is gathered, both
// launches take 9 us for 3000 tokens, 16 for 16 x 4 heads of up to 32768.  Keys past the
// registers cost a load each in every pass, one behind the other: 78 us for 16 x 4 heads of
// 131072.  (A byte at a time with the digit found by one thread, a CTA to a pair: 26 and 43
// for this launch alone; the keys of the first digit's bin listed for the other two: no
// change.)
template <int CTAS>
__global__ __launch_bounds__(kThreads) void evict_select_kernel(KvView kv, EvictArgs a, unsigned* err) {
  __shared__ uint32_t s_hist[3][kBins];  // one for each digit
  __shared__ uint32_t s_sums[2][kWarps];
  __shared__ uint32_t s_found[3][2];     // digit, keys above it, keys in it
  __shared__ uint32_t s_size[3];
  __shared__ int s_above[kWarps], s_same[kWarps], s_counts[2];
  const cg::cluster_group cluster = cg::this_cluster();
  const auto meet = [&]() {  // the pair's CTAs
    if constexpr (CTAS == 1)
      __syncthreads();
    else
      cluster.sync();
  };
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t pair = blockIdx.x / CTAS;
  const int rank = static_cast<int>(blockIdx.x % CTAS);
  const int b = static_cast<int>(pair / kv.hkv);
  const int64_t most = static_cast<int64_t>(kv.max_blocks) * kv.block;
  int L = max(__ldg(kv.seq_lens + b), 0);
  if (L > most) {
    if (tid == 0 && rank == 0) set_error(err, HS_EBIT_BLOCK_RANGE);
    L = static_cast<int>(most);
  }
  int32_t* kept = a.kept + pair * a.budget;
  constexpr int all = CTAS * kThreads;
  const int me = rank * kThreads + tid;
  if (L <= a.budget) {  // (the same for the whole cluster)
    for (int i = me; i < a.budget; i += all) kept[i] = i < L ? i : -1;
    return;
  }
  const int first = a.sink, last = L - a.recent;  // the tokens that are chosen from
  const int need = a.budget - a.sink - a.recent;
  for (int i = me; i < a.sink; i += all) kept[i] = i;
  for (int i = me; i < a.recent; i += all) kept[a.budget - a.recent + i] = last + i;
  if (need == 0) return;
  const float* w = a.weights + pair * most;
  // this warp's run, lane i every 32nd token of it
  const int turns = ((last - first + CTAS * kWarps - 1) / (CTAS * kWarps) + 31) / 32;
  const int64_t run0 = first + static_cast<int64_t>(rank * kWarps + warp) * turns * 32;
  const int t0 = static_cast<int>(min(static_cast<int64_t>(last), run0)), n = min(turns * 32, last - t0);
  // (loads behind conditions would wait for each other: places past the run read its last)
  float raw[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) raw[i] = __ldg(w + min(t0 + 32 * i + lane, last - 1));
  uint32_t held[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) held[i] = weight_key(raw[i]);
  // each(turn, key, there) over the run
  const auto over = [&](auto&& each) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      if (32 * i >= n) return;
      each(i, held[i], 32 * i + lane < n);
    }
    for (int i = kHeld; 32 * i < n; ++i) {
      const bool there = 32 * i + lane < n;
      each(i, there ? weight_key(__ldg(w + t0 + 32 * i + lane)) : 0u, there);
    }
  };
  for (int i = tid; i < 3 * kBins; i += kThreads) (&s_hist[0][0])[i] = 0u;
  __syncthreads();
  // ---- the key of the last that stays: its digits, and how many of that key do ----
  uint32_t prefix = 0u, mask = 0u;
  int rest = need;  // of the keys that share the digits so far
  bool all_stay = false;  // all of them
#pragma unroll 1
  for (int digit = 0; digit < 3; ++digit) {
    const int shift = digit == 0 ? 21 : digit == 1 ? 10 : 0;
    const uint32_t field = digit == 2 ? 1023u : 2047u;
    over([&](int, uint32_t k, bool there) {
      if (there && (k & mask) == prefix) atomicAdd(&s_hist[digit][(k >> shift) & field], 1u);
    });
    meet();
    // bins 2047 - 2 tid and 2046 - 2 tid of the cluster, from the largest down
    uint32_t h[2] = {0u, 0u};
#pragma unroll
    for (int c = 0; c < CTAS; ++c) {
      const uint2 two = CTAS == 1 ? *reinterpret_cast<const uint2*>(&s_hist[digit][kBins - 2 - 2 * tid]) : *reinterpret_cast<const uint2*>(cluster.map_shared_rank(&s_hist[digit][0], c) + kBins - 2 - 2 * tid);
      h[0] += two.y;
      h[1] += two.x;
    }
    uint32_t incl = h[0] + h[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) s_sums[digit & 1][warp] = incl;
    __syncthreads();
    uint32_t before = lane < warp ? s_sums[digit & 1][lane] : 0u;
    before = __reduce_add_sync(0xffffffffu, before);
    uint32_t above = before + incl - h[0] - h[1];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (above < static_cast<uint32_t>(rest) && static_cast<uint32_t>(rest) <= above + h[i]) {
        s_found[digit][0] = kBins - 1 - 2 * tid - i;
        s_found[digit][1] = above;
        s_size[digit] = h[i];
      }
      above += h[i];
    }
    __syncthreads();
    prefix |= s_found[digit][0] << shift;
    mask |= field << shift;
    rest -= static_cast<int>(s_found[digit][1]);
    all_stay = s_size[digit] == static_cast<uint32_t>(rest);
    if (all_stay) break;
  }
  // ---- the indices in order: keys from `from` on, and, but where all stay, the first
  // `rest` whose digits are the same (no key has the largest digits: no overflow) ----
  const uint32_t from = all_stay ? prefix : (prefix | ~mask) + 1u;
  int above = 0, same = 0;
  over([&](int, uint32_t k, bool there) {
    above += there && k >= from;
    same += there && !all_stay && (k & mask) == prefix;
  });
  above = __reduce_add_sync(0xffffffffu, above);
  same = __reduce_add_sync(0xffffffffu, same);
  if (lane == 0) {
    s_above[warp] = above;
    s_same[warp] = same;
  }
  __syncthreads();
  const int wa = s_above[lane], ws = s_same[lane];
  above = __reduce_add_sync(0xffffffffu, lane < warp ? wa : 0);  // of the warps before
  same = __reduce_add_sync(0xffffffffu, lane < warp ? ws : 0);
  if (warp == 0) {
    const int ca = __reduce_add_sync(0xffffffffu, wa), cs = __reduce_add_sync(0xffffffffu, ws);
    if (lane == 0) {
      s_counts[0] = ca;
      s_counts[1] = cs;
    }
  }
  meet();
  for (int c = 0; c < rank; ++c) {
    const int* counts = cluster.map_shared_rank(s_counts, c);
    above += counts[0];
    same += counts[1];
  }
  const unsigned lower = (1u << lane) - 1u;
  int32_t* mine = kept + a.sink;
  if (all_stay) {
    over([&](int i, uint32_t k, bool there) {
      const bool stays = there && k >= from;
      const unsigned m = __ballot_sync(0xffffffffu, stays);
      if (stays) mine[above + __popc(m & lower)] = t0 + 32 * i + lane;
      above += __popc(m);
    });
  } else {
    over([&](int i, uint32_t k, bool there) {
      const bool is_above = there && k >= from, is_same = there && (k & mask) == prefix;
      const unsigned ma = __ballot_sync(0xffffffffu, is_above), ms = __ballot_sync(0xffffffffu, is_same);
      const int same_here = same + __popc(ms & lower), above_here = above + __popc(ma & lower);
      if (is_above || (is_same && same_here < rest)) mine[above_here + min(same_here, rest)] = t0 + 32 * i + lane;
      above += __popc(ma);
      same += __popc(ms);
    });
  }
  if constexpr (CTAS > 1) cluster.sync();  // no CTA leaves while another reads its shared memory
}

constexpr int kRows = 64;  // rows of a CTA
constexpr int kGatherThreads = 256;
constexpr int kFlight = 4;  // pieces of a thread on their way

// CTA = kRows places of a (request, kv head)'s new pages.  row_bytes, scale_bytes: of a
// row of K (or V).  Memory-bound: 16 x 4 heads, 4096 rows each of 512 bytes of K and V,
// 268 MB: 41 us, the copy rate; rows of 128 and 64 bytes, scattered, half of it.
__global__ __launch_bounds__(kGatherThreads) void evict_gather_kernel(KvView kv, KvView dst, EvictArgs a, int chunks, int row_bytes,
                                                                      int scale_bytes, int scale_unit, unsigned* err) {
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
  const int pieces = row_bytes / 16, each = pieces * 2;  // (a power of two)
  const int shift = 31 - __clz(each);
  for (int n0 = tid; n0 < kRows * each; n0 += kFlight * kGatherThreads) {
    uint4 x[kFlight];
    char* to[kFlight];
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      const int n = n0 + u * kGatherThreads, r = n >> shift, c = n - (r << shift);
      to[u] = nullptr;
      if (n >= kRows * each || s_from[r] < 0) continue;
      const bool v = c >= pieces;
      const int at = (v ? c - pieces : c) * 16;
      x[u] = __ldg(reinterpret_cast<const uint4*>(static_cast<const char*>(v ? kv.v_pages : kv.k_pages) + s_from[r] * row_bytes + at));
      to[u] = static_cast<char*>(const_cast<void*>(v ? dst.v_pages : dst.k_pages)) + s_to[r] * row_bytes + at;
    }
#pragma unroll
    for (int u = 0; u < kFlight; ++u)
      if (to[u]) *reinterpret_cast<uint4*>(to[u]) = x[u];
  }
  // scales, by the widest units that their rows and addresses allow
  const auto copy_scales = [&](auto unit) {
    using Unit = decltype(unit);
    const int n_row = scale_bytes / static_cast<int>(sizeof(Unit));
    for (int n = tid; n < kRows * n_row * 2; n += kGatherThreads) {
      const int r = n / (n_row * 2), x = n - r * n_row * 2;
      const bool v = x >= n_row;
      const int at = v ? x - n_row : x;
      if (s_from[r] < 0) continue;
      const Unit* src = reinterpret_cast<const Unit*>(v ? kv.v_scales : kv.k_scales) + s_from[r] * n_row + at;
      Unit* to = reinterpret_cast<Unit*>(const_cast<float*>(v ? dst.v_scales : dst.k_scales)) + s_to[r] * n_row + at;
      *to = __ldg(src);
    }
  };
  if (scale_unit == 16)
    copy_scales(uint4{});
  else if (scale_unit == 8)
    copy_scales(uint2{});
  else if (scale_unit == 4)
    copy_scales(uint32_t{});
}

template <int CTAS>
cudaError_t launch_select_by(const KvView& kv, const EvictArgs& a, unsigned* err, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(static_cast<int64_t>(kv.batch) * kv.hkv * CTAS));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CTAS;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, evict_select_kernel<CTAS>, kv, a, err);
}
cudaError_t launch_select(const KvView& kv, const EvictArgs& a, int sms, unsigned* err, cudaStream_t st) {
  const int64_t pairs = static_cast<int64_t>(kv.batch) * kv.hkv, tokens = static_cast<int64_t>(kv.max_blocks) * kv.block;
  // as many CTAs to a pair as keep its longest request's keys in registers, four to a
  // thread where there is room, and as all pairs leave room for at once (one on an SM)
  int ctas = 1;
  while (ctas < kMostCtas && tokens > static_cast<int64_t>(ctas) * kThreads * 4 && pairs * 2 * ctas <= sms) ctas *= 2;
  switch (ctas) {
    case 1: return launch_select_by<1>(kv, a, err, st);
    case 2: return launch_select_by<2>(kv, a, err, st);
    case 4: return launch_select_by<4>(kv, a, err, st);
    default: return launch_select_by<kMostCtas>(kv, a, err, st);
  }
}

}  // namespace

int64_t evict_ctas(const KvView& kv, int budget) {
  return static_cast<int64_t>(kv.batch) * kv.hkv * ceil_div(budget, kRows);
}

cudaError_t launch_evict(const KvView& kv, const KvView& dst, const EvictArgs& a, int sms, unsigned* err, cudaStream_t st) {
  if (kv.batch == 0) return cudaSuccess;
  cudaError_t e = launch_select(kv, a, sms, err, st);
  if (e != cudaSuccess) return e;
  const int elem2 = kv.kv_dtype == HS_KV_F32 ? 8 : kv.kv_dtype == HS_KV_BF16 ? 4 : kv.kv_dtype == HS_KV_INT4_G32 ? 1 : 2;
  const int scale_bytes = kv.kv_dtype >= HS_KV_FP8E4M3_G32 ? kv.head_dim / kQuantGroup * 4 : 0;
  const uintptr_t bases = reinterpret_cast<uintptr_t>(kv.k_scales) | reinterpret_cast<uintptr_t>(kv.v_scales) |
                          reinterpret_cast<uintptr_t>(dst.k_scales) | reinterpret_cast<uintptr_t>(dst.v_scales);
  const int scale_unit = scale_bytes == 0 ? 0 : bases % scale_bytes == 0 ? scale_bytes : 4;
  return launch_pdl(evict_gather_kernel, dim3(static_cast<unsigned>(evict_ctas(kv, a.budget))), dim3(kGatherThreads), 0, st, kv, dst, a,
                    ceil_div(a.budget, kRows), kv.head_dim * elem2 / 2, scale_bytes, scale_unit, err);
}

}  // namespace hs
