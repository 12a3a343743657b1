// k_route.cu -- the router of the sparse MLP block: for every token the k
// experts with the largest logits, their softmax weights, and the order of
// the (token, expert) entries by expert that the grouped products read.
//
//     p[t,e] = exp(l[t,e] - max_e l) / sum_e exp(l[t,e] - max_e l)
//     ids[t,j]     = expert of the j-th largest logit (ties: lowest number)
//     weights[t,j] = scale * p, or scale * p / (sum of the chosen p)
//     rows, slots  = the entries (t, j) in the order (expert, t k + j)
//
// One warp per token: lane l holds the logits of experts l, l + 32, ..., as
// 32-bit keys whose unsigned order is the floats' order (0 = no expert: a
// masked logit of -inf or a lane past E).  One round per choice: a warp
// maximum of the keys, then a warp minimum of the expert numbers that hold
// it, so ties need no second pass.
//
// The order is a counting sort that keeps entries in sequence, without
// atomics, so its result does not depend on timing: each warp counts its own
// tokens' entries by expert (equal experts within 32 entries are found with
// match_any), the warps' counts are summed in order, and each warp walks its
// entries again and numbers them.
//
// Up to kOneTokens tokens one block does all of it in one launch.  Beyond
// that a first kernel chooses and counts per block of tokens (counts go to
// the workspace) and a second one, overlapped by programmatic dependent
// launch, sums the counts of the blocks before its own and numbers its
// entries.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "launch.h"
#include "sm103_ptx.cuh"
#include "swiglu.h"

namespace swiglu {
namespace {

constexpr int kMaxE = 1024;
constexpr int kMaxK = 32;
constexpr int kWarps = 16;               // warps per block
constexpr int kThreads = 32 * kWarps;
constexpr int kBlockTokens = 128;        // tokens per block, several blocks
constexpr int kOneTokens = 128;          // tokens of the one-block form
constexpr unsigned kAll = 0xffffffffu;

struct RouteParams {
  const void *logits;
  int32_t *ids;
  float *weights;
  int32_t *offsets, *rows, *slots;
  int32_t *counts;  // [blocks][E], several blocks only
  int32_t T, E, k, blocks;
  int32_t renormalize;
  float scale;
};

// Unsigned key with the order of the floats; -inf -> 0 (masked), NaN above
// +inf (it is chosen first and its weight comes out NaN, so it stays visible).
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x == -INFINITY) return 0u;
  if (x != x) return 0xffffffffu;
  if (x == 0.0f) return 0x80000000u;  // both zeros
  const uint32_t b = __float_as_uint(x);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float key_value(uint32_t key) {
  if (key == 0xffffffffu) return NAN;
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7fffffffu) : ~key);
}

__device__ __forceinline__ float warp_total(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// One token by one warp; the chosen experts go to `ids16` (shared; 0xffff =
// none) and to global memory.
template <int EPL, bool FP32>
__device__ __forceinline__ void choose(const RouteParams &p, int t, int lane, uint16_t *ids16) {
  uint32_t key[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 32 * i;
    key[i] = 0u;
    if (e < p.E) {
      const int64_t at = int64_t(t) * p.E + e;
      key[i] = order_key(FP32 ? __ldg(static_cast<const float *>(p.logits) + at)
                              : __bfloat162float(static_cast<const __nv_bfloat16 *>(p.logits)[at]));
    }
  }
  uint32_t best = 0u;
#pragma unroll
  for (int i = 0; i < EPL; ++i) best = max(best, key[i]);
  const uint32_t top = __reduce_max_sync(kAll, best);
  const float m = key_value(top);
  float sum = 0.0f;
  if (!p.renormalize && top != 0u) {
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (key[i] != 0u) sum += expf(key_value(key[i]) - m);
    sum = warp_total(sum);
  }
  int my_id = -1;       // lane j keeps choice j
  float my_e = 0.0f;
  for (int j = 0; j < p.k; ++j) {
    const uint32_t mx = j == 0 ? top : __reduce_max_sync(kAll, best);
    if (mx == 0u) break;
    uint32_t at = 0xffffffffu;
    if (best == mx) {
#pragma unroll
      for (int i = EPL - 1; i >= 0; --i)
        if (key[i] == mx) at = lane + 32 * i;
    }
    const uint32_t e = __reduce_min_sync(kAll, at);
    if (lane == j) {
      my_id = static_cast<int>(e);
      my_e = expf(key_value(mx) - m);
    }
    if (at == e) {  // the owner takes it out
      best = 0u;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        if (lane + 32 * i == static_cast<int>(e)) key[i] = 0u;
        best = max(best, key[i]);
      }
    }
  }
  if (p.renormalize) sum = warp_total(my_e);
  if (lane < p.k) {
    const int64_t at = int64_t(t) * p.k + lane;
    p.ids[at] = my_id;
    p.weights[at] = my_id < 0 ? 0.0f : p.scale * (my_e / sum);
    ids16[lane] = my_id < 0 ? uint16_t(0xffff) : uint16_t(my_id);
  }
}

// Walks this warp's entries [i0, i1) of the block, 32 at a time.  NUMBER =
// false: counts them into cnt[expert]; true: cnt[expert] holds the number of
// entries of the block before this warp's, and each entry gets its place.
template <bool NUMBER>
__device__ __forceinline__ void walk(const RouteParams &p, const uint16_t *ids16, int i0, int i1,
                                     uint16_t *cnt, const int32_t *base, int t0, int lane) {
  for (int b = i0; b < i1; b += 32) {
    const int i = b + lane;
    const unsigned e = i < i1 ? ids16[i] : 0xffffu;
    const unsigned same = __match_any_sync(kAll, e);
    const unsigned before = same & ((1u << lane) - 1u);
    if (NUMBER && i < i1) {
      const int64_t entry = int64_t(t0) * p.k + i;
      if (e != 0xffffu) {
        const int pos = base[e] + cnt[e] + __popc(before);
        p.slots[entry] = pos;
        p.rows[pos] = static_cast<int32_t>(entry / p.k);
      } else {
        p.slots[entry] = -1;
      }
    }
    __syncwarp();
    if (e != 0xffffu && before == 0u) cnt[e] += static_cast<uint16_t>(__popc(same));
    __syncwarp();
  }
}

struct RouteSmem {
  uint16_t cnt[kWarps][kMaxE];
  int32_t base[kMaxE];
  uint16_t ids[kBlockTokens * kMaxK];
  int32_t carry[33];
};

// Replaces v (one value per thread; thread i < n holds element i) by the sum
// of the elements before it; `total` gets the sum.  All threads.
__device__ __forceinline__ int block_exclusive_scan(int v, int32_t *carry, int &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int w = __shfl_up_sync(kAll, s, o);
    if (lane >= o) s += w;
  }
  if (lane == 31) carry[warp] = s;
  __syncthreads();
  if (warp == 0) {
    int c = lane < kWarps ? carry[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int w = __shfl_up_sync(kAll, c, o);
      if (lane >= o) c += w;
    }
    carry[lane] = c;
  }
  __syncthreads();
  const int before = warp > 0 ? carry[warp - 1] : 0;
  total = carry[kWarps - 1];
  __syncthreads();
  return before + s - v;
}

// cnt[w][e] -> entries of the block's warps before w; returns the block's
// count of each of this thread's experts through `counted(e, n)`.
template <class F>
__device__ __forceinline__ void scan_warps(RouteSmem &sm, int E, F counted) {
  for (int e = threadIdx.x; e < E; e += kThreads) {
    int run = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const int c = sm.cnt[w][e];
      sm.cnt[w][e] = static_cast<uint16_t>(run);
      run += c;
    }
    counted(e, run);
  }
}

__device__ __forceinline__ void clear_counts(RouteSmem &sm, int E) {
  for (int i = threadIdx.x; i < kWarps * E; i += kThreads) sm.cnt[i / E][i % E] = 0;
}

// base[e] (the count of expert e) -> first place of expert e, for all E
// experts; returns the number of routed entries.
__device__ __forceinline__ int scan_experts(RouteSmem &sm, int E, int32_t *offsets) {
  int carried = 0;
  for (int e0 = 0; e0 < E; e0 += kThreads) {
    const int e = e0 + threadIdx.x;
    int total;
    const int before = block_exclusive_scan(e < E ? sm.base[e] : 0, sm.carry, total);
    if (e < E) {
      sm.base[e] = carried + before;
      if (offsets) offsets[e] = carried + before;
    }
    carried += total;
  }
  if (offsets && threadIdx.x == 0) offsets[E] = carried;
  return carried;
}

// Everything in one block.
template <int EPL, bool FP32>
__global__ void __launch_bounds__(kThreads) route_one_kernel(const RouteParams p) {
  __shared__ RouteSmem sm;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  ptx::grid_launch_dependents();
  clear_counts(sm, p.E);
  ptx::grid_dependency_wait();
  const int per = (p.T + kWarps - 1) / kWarps;
  const int t0 = min(warp * per, p.T), t1 = min(t0 + per, p.T);
  for (int t = t0; t < t1; ++t) choose<EPL, FP32>(p, t, lane, sm.ids + t * p.k);
  __syncthreads();
  walk<false>(p, sm.ids, t0 * p.k, t1 * p.k, sm.cnt[warp], nullptr, 0, lane);
  __syncthreads();
  scan_warps(sm, p.E, [&](int e, int n) { sm.base[e] = n; });
  __syncthreads();
  const int routed = scan_experts(sm, p.E, p.offsets);
  __syncthreads();
  walk<true>(p, sm.ids, t0 * p.k, t1 * p.k, sm.cnt[warp], sm.base, 0, lane);
  for (int i = routed + threadIdx.x; i < p.T * p.k; i += kThreads) p.rows[i] = -1;
}

// Several blocks, first pass: choose, and count the block's entries.
template <int EPL, bool FP32>
__global__ void __launch_bounds__(kThreads) route_choose_kernel(const RouteParams p) {
  __shared__ RouteSmem sm;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  ptx::grid_launch_dependents();
  clear_counts(sm, p.E);
  ptx::grid_dependency_wait();
  const int b0 = blockIdx.x * kBlockTokens, nt = min(kBlockTokens, p.T - b0);
  const int per = (nt + kWarps - 1) / kWarps;
  const int t0 = min(warp * per, nt), t1 = min(t0 + per, nt);
  for (int t = t0; t < t1; ++t) choose<EPL, FP32>(p, b0 + t, lane, sm.ids + t * p.k);
  __syncthreads();
  walk<false>(p, sm.ids, t0 * p.k, t1 * p.k, sm.cnt[warp], nullptr, 0, lane);
  __syncthreads();
  scan_warps(sm, p.E, [&](int e, int n) { p.counts[int64_t(blockIdx.x) * p.E + e] = n; });
}

// Several blocks, second pass: places of the block's entries.
__global__ void __launch_bounds__(kThreads) route_order_kernel(const RouteParams p) {
  __shared__ RouteSmem sm;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.x;
  ptx::grid_launch_dependents();
  clear_counts(sm, p.E);
  int32_t *mine = reinterpret_cast<int32_t *>(sm.ids);  // [E] entries of the blocks before this one
  for (int e = threadIdx.x; e < p.E; e += kThreads) {
    sm.base[e] = 0;
    mine[e] = 0;
  }
  ptx::grid_dependency_wait();
  __syncthreads();
  // Counts of every block: thread (g, e) sums blocks g, g + G, ... (integer
  // sums in shared memory: their order does not matter).
  const int G = max(1, kThreads / p.E);
  for (int e0 = 0; e0 < p.E; e0 += kThreads) {
    const int e = e0 + (p.E >= kThreads ? static_cast<int>(threadIdx.x) : static_cast<int>(threadIdx.x) % p.E);
    const int g = p.E >= kThreads ? 0 : threadIdx.x / p.E;
    if (e < p.E && g < G) {
      int all = 0, before = 0;
#pragma unroll 8
      for (int i = g; i < p.blocks; i += G) {
        const int c = __ldg(p.counts + int64_t(i) * p.E + e);
        all += c;
        before += i < b ? c : 0;
      }
      atomicAdd(&sm.base[e], all);
      atomicAdd(&mine[e], before);
    }
  }
  __syncthreads();
  const int routed = scan_experts(sm, p.E, b == 0 ? p.offsets : nullptr);
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += kThreads) sm.base[e] += mine[e];
  __syncthreads();
  const int b0 = b * kBlockTokens, nt = min(kBlockTokens, p.T - b0);
  for (int i = threadIdx.x; i < nt * p.k; i += kThreads)
    sm.ids[i] = static_cast<uint16_t>(__ldg(p.ids + int64_t(b0) * p.k + i));  // -1 -> 0xffff
  __syncthreads();
  const int per = (nt + kWarps - 1) / kWarps;
  const int t0 = min(warp * per, nt), t1 = min(t0 + per, nt);
  walk<false>(p, sm.ids, t0 * p.k, t1 * p.k, sm.cnt[warp], nullptr, b0, lane);
  __syncthreads();
  scan_warps(sm, p.E, [](int, int) {});
  __syncthreads();
  walk<true>(p, sm.ids, t0 * p.k, t1 * p.k, sm.cnt[warp], sm.base, b0, lane);
  const int64_t entries = int64_t(p.T) * p.k;
  for (int64_t i = routed + int64_t(b) * kThreads + threadIdx.x; i < entries;
       i += int64_t(p.blocks) * kThreads)
    p.rows[i] = -1;
}

cudaError_t launch_pdl(void (*kern)(RouteParams), int grid, const RouteParams &p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int EPL>
cudaError_t launch_route(bool fp32, const RouteParams &p, cudaStream_t s) {
  if (p.T <= kOneTokens)
    return launch_pdl(fp32 ? route_one_kernel<EPL, true> : route_one_kernel<EPL, false>, 1, p, s);
  cudaError_t e = launch_pdl(fp32 ? route_choose_kernel<EPL, true> : route_choose_kernel<EPL, false>,
                             p.blocks, p, s);
  return e != cudaSuccess ? e : launch_pdl(route_order_kernel, p.blocks, p, s);
}

}  // namespace
}  // namespace swiglu

extern "C" uint64_t swiglu_moe_route_workspace_size(int64_t T, int64_t E, int64_t k) {
  using namespace swiglu;
  if (T <= kOneTokens || E < 1 || k < 1) return 0;
  return uint64_t((T + kBlockTokens - 1) / kBlockTokens) * E * 4;
}

extern "C" int swiglu_moe_route(const void *logits, int32_t logits_fp32, int32_t renormalize,
                                float scale, int32_t *ids, float *weights, int32_t *offsets,
                                int32_t *rows, int32_t *slots, int64_t T, int64_t E, int64_t k,
                                void *workspace, uint64_t workspace_bytes, void *stream) {
  using namespace swiglu;
  if (T < 0 || E < 1 || k < 1 || k > E || (logits_fp32 != 0 && logits_fp32 != 1) ||
      (renormalize != 0 && renormalize != 1) || !std::isfinite(scale))
    return SWIGLU_ERR_INVALID_ARG;
  const int64_t limit = (int64_t(1) << 31) - 1;
  if (E > kMaxE || k > kMaxK || T > limit / k) return SWIGLU_ERR_UNSUPPORTED;
  if (!offsets || (T > 0 && (!logits || !ids || !weights || !rows || !slots)))
    return SWIGLU_ERR_INVALID_ARG;
  if (!ptr_aligned(logits, logits_fp32 ? 4 : 2) || !ptr_aligned(ids, 4) || !ptr_aligned(weights, 4) ||
      !ptr_aligned(offsets, 4) || !ptr_aligned(rows, 4) || !ptr_aligned(slots, 4) ||
      !ptr_aligned(workspace, 4))
    return SWIGLU_ERR_MISALIGNED;
  const uint64_t need = swiglu_moe_route_workspace_size(T, E, k);
  if (need > 0 && (!workspace || workspace_bytes < need)) return SWIGLU_ERR_INVALID_ARG;
  // no output may overlap the logits, the workspace or another output
  const uint64_t n4 = uint64_t(T) * k * 4;
  const void *ptr[7] = {logits, ids, weights, rows, slots, offsets, need ? workspace : nullptr};
  const uint64_t len[7] = {uint64_t(T) * E * (logits_fp32 ? 4 : 2), n4, n4, n4, n4,
                           uint64_t(E + 1) * 4, need};
  for (int i = 0; i < 7; ++i)
    for (int j = 0; j < i; ++j)
      if (ranges_overlap(ptr[i], len[i], ptr[j], len[j])) return SWIGLU_ERR_INVALID_ARG;
  uint32_t *err = nullptr;
  int sms = 0;
  uint64_t timeout_ns = 0, gen = 0;
  int rc = device_info(&err, &sms, &timeout_ns, &gen);
  if (rc != SWIGLU_OK) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0)
    return cudaMemsetAsync(offsets, 0, uint64_t(E + 1) * 4, s) == cudaSuccess ? SWIGLU_OK
                                                                              : SWIGLU_ERR_CUDA;
  RouteParams p;
  p.logits = logits;
  p.ids = ids;
  p.weights = weights;
  p.offsets = offsets;
  p.rows = rows;
  p.slots = slots;
  p.counts = static_cast<int32_t *>(workspace);
  p.T = int32_t(T);
  p.E = int32_t(E);
  p.k = int32_t(k);
  p.blocks = int32_t((T + kBlockTokens - 1) / kBlockTokens);
  p.renormalize = renormalize;
  p.scale = scale;
  const bool f = logits_fp32 != 0;
  const cudaError_t e = E <= 32    ? launch_route<1>(f, p, s)
                        : E <= 64  ? launch_route<2>(f, p, s)
                        : E <= 128 ? launch_route<4>(f, p, s)
                        : E <= 256 ? launch_route<8>(f, p, s)
                        : E <= 512 ? launch_route<16>(f, p, s)
                                   : launch_route<32>(f, p, s);
  return e == cudaSuccess ? SWIGLU_OK : SWIGLU_ERR_CUDA;
}
