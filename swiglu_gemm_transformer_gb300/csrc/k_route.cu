// k_route.cu -- the router of the sparse MLP block: for every token the k
// experts with the largest logits, their softmax weights, and the order of
// the (token, expert) entries by expert that the grouped products read.
//
//     p[t,e] = exp(l[t,e] - max_e l) / sum_e exp(l[t,e] - max_e l)
//     ids[t,j]     = expert of the j-th largest logit (ties: lowest number)
//     weights[t,j] = scale * p, or scale * p / (sum of the chosen p)
//     rows, slots  = the entries (t, j) in the order (expert, t k + j)
//
// LPT lanes per token (4 to 32: at least k, and eight experts a lane while that
// is enough): lane l holds the logits of experts l, l + LPT, ... as 32-bit keys
// whose unsigned order is the floats' order.  A key of 0 is no expert: a masked
// logit of -inf, or a lane past E.  A choice is one maximum over the group's
// lanes (log2(LPT) shuffles) of the key with the complement of the expert's
// number below it, so that among equal logits the lowest number wins.  What
// counts is the length of this chain (k rounds of it, each on the one before),
// so nothing in it branches.
//
// The order is a counting sort that keeps entries in sequence, without
// atomics, so its result does not depend on timing: each warp counts its own
// tokens' entries by expert (equal experts within 32 entries are found with
// match_any), the warps' counts are summed in order, and each warp walks its
// entries again and numbers them within the block.
//
// Up to kOneTokens tokens are one launch of one cluster, 32 tokens a block: one
// SM issues the choices of 128 tokens in about 6 us, so a few tokens are spread
// over several; the blocks read each other's counts through distributed shared
// memory (128 tokens: 5.4 us, in one block 9.1 us).  Beyond that a first kernel
// numbers the entries within each block of 32 to 128 tokens (in slots) and writes
// the block's counts to the workspace, and a second one, overlapped by
// programmatic dependent launch, sums the counts of the blocks before its own
// and adds them (16384 tokens: 14.0 us; in clusters of eight blocks of 32
// tokens about a fifth more).  Every block of the second launch reads the counts
// of all blocks, which is little at such sizes but grows with the square of the
// tokens: 131072 tokens take 100 us with 64 experts and 292 us with 256.
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
constexpr int kOneTokens = 256;          // tokens of the one-launch form,
constexpr int kOneBlockTokens = 32;      // per block of its cluster (at most eight)
constexpr int kBlockTokens = 128;        // most tokens per block otherwise
// Warps of a block x experts: 32 warps up to 510 experts, and RouteSmem is the 48 KB
// that a kernel may hold without asking.
constexpr int kCounters = 16320;
constexpr unsigned kAll = 0xffffffffu;

struct RouteParams {
  const void *logits;
  int32_t *ids;
  float *weights;
  int32_t *offsets, *rows, *slots;
  int32_t *counts;  // [blocks][E], two launches only
  int32_t T, E, k, blocks, block_tokens;
  int32_t renormalize;
  float scale;
};

// Unsigned number with the order of the floats; -inf -> 0 (masked), NaN above
// +inf (it is chosen first and its weight comes out NaN, so it stays visible).
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(__fadd_rn(x, 0.0f));  // -0 becomes +0
  const uint32_t k = b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
  return x != x ? 0xffffffffu : k == 0x007fffffu ? 0u : k;
}

__device__ __forceinline__ float key_value(uint32_t key) {
  const uint32_t b = key ^ ((key & 0x80000000u) ? 0x80000000u : 0xffffffffu);
  return key == 0u ? -INFINITY : __uint_as_float(b);  // all ones -> a NaN
}

// The token t of this lane's group of LPT >= k lanes (or none: t >= end), its
// chosen experts to ids16 (shared; 0xffff = none) and global memory.  All
// lanes of the warp call it together.
template <int LPT, int EPL, bool FP32>
__device__ __forceinline__ void choose(const RouteParams &p, int64_t t, int64_t end, int lane,
                                       uint16_t *ids16) {
  using Pick = unsigned long long;  // key above ~expert; 0 in the upper half: none
  const int l = lane & (LPT - 1);
  const bool live = t < end;
  float x[EPL];
  uint32_t key[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = l + LPT * i;
    x[i] = -INFINITY;
    if (live && e < p.E) {
      const int64_t at = t * p.E + e;
      x[i] = FP32 ? __ldg(static_cast<const float *>(p.logits) + at)
                  : __bfloat162float(static_cast<const __nv_bfloat16 *>(p.logits)[at]);
    }
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) key[i] = order_key(x[i]);
  // this lane's largest key, the first that holds it
  auto best = [&]() {
    uint32_t b[EPL];
    int w[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) b[i] = key[i], w[i] = i;
#pragma unroll
    for (int st = 1; st < EPL; st <<= 1)
#pragma unroll
      for (int i = 0; i + st < EPL; i += 2 * st) {
        const bool up = b[i + st] > b[i];
        b[i] = up ? b[i + st] : b[i];
        w[i] = up ? w[i + st] : w[i];
      }
    return (Pick(b[0]) << 32) | ~static_cast<uint32_t>(l + LPT * w[0]);
  };
  auto group_max = [](Pick v) {
#pragma unroll
    for (int o = LPT / 2; o > 0; o >>= 1) {
      const Pick u = __shfl_xor_sync(kAll, v, o);
      v = u > v ? u : v;
    }
    return v;
  };
  Pick mx = group_max(best());
  const float m = key_value(static_cast<uint32_t>(mx >> 32));
  float sum = 0.0f;
  if (!p.renormalize) {
    // a masked logit adds exp(-inf) = 0 (where all are, the sum is not used)
#pragma unroll
    for (int i = 0; i < EPL; ++i) sum += expf(x[i] - m);
  }
  uint32_t my_key = 0u;  // lane j of the group keeps choice j
  int my_id = -1;
  for (int j = 0; j < p.k; ++j) {
    const uint32_t top = static_cast<uint32_t>(mx >> 32);
    const int e = top != 0u ? static_cast<int>(~static_cast<uint32_t>(mx)) : -1;
    my_key = l == j ? top : my_key;
    my_id = l == j ? e : my_id;
#pragma unroll
    for (int i = 0; i < EPL; ++i) key[i] = l + LPT * i == e ? 0u : key[i];
    mx = group_max(best());
  }
  const float w = my_id < 0 ? 0.0f : expf(key_value(my_key) - m);
  sum = p.renormalize ? w : sum;
#pragma unroll
  for (int o = LPT / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
  if (live && l < p.k) {
    p.ids[t * p.k + l] = my_id;
    p.weights[t * p.k + l] = my_id < 0 ? 0.0f : p.scale * (w / sum);
    ids16[l] = static_cast<uint16_t>(my_id);  // -1 -> 0xffff
  }
}

// Walks this warp's entries [i0, i1) of the block, 32 at a time, adding them to
// cnt[expert]; number(i, e, before) gets each entry's expert and the entries
// counted before it (e = 0xffff: none).
template <class F>
__device__ __forceinline__ void walk(const uint16_t *ids16, int i0, int i1, uint16_t *cnt, int lane,
                                     F number) {
  for (int b = i0; b < i1; b += 32) {
    const int i = b + lane;
    const unsigned e = i < i1 ? ids16[i] : 0xffffu;
    const unsigned same = __match_any_sync(kAll, e);
    const unsigned before = same & ((1u << lane) - 1u);
    if (i < i1) number(i, e, e != 0xffffu ? cnt[e] + __popc(before) : 0);
    __syncwarp();
    if (e != 0xffffu && before == 0u) cnt[e] += static_cast<uint16_t>(__popc(same));
    __syncwarp();
  }
}

struct RouteSmem {
  uint16_t cnt[kCounters];  // [warp][E]
  int32_t base[kMaxE];      // first place of each expert's entries
  int32_t total[kMaxE];     // entries of this block (read by the cluster's other blocks), or of the blocks before
  uint16_t ids[kBlockTokens * kMaxK];
  int32_t carry[32];
};

static_assert(sizeof(RouteSmem) <= 48 * 1024, "static shared memory");

// Exclusive scan of base[0, E) in place; returns the total.  All threads.
__device__ __forceinline__ int scan_experts(RouteSmem &sm, int E, int32_t *offsets) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int carried = 0;
  for (int e0 = 0; e0 < E; e0 += blockDim.x) {
    const int e = e0 + threadIdx.x;
    const int v = e < E ? sm.base[e] : 0;
    int s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int w = __shfl_up_sync(kAll, s, o);
      if (lane >= o) s += w;
    }
    if (lane == 31) sm.carry[warp] = s;
    __syncthreads();
    int c = lane < warps ? sm.carry[lane] : 0;  // every warp scans the warps' sums
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int w = __shfl_up_sync(kAll, c, o);
      if (lane >= o) c += w;
    }
    const int before = __shfl_sync(kAll, c, max(warp - 1, 0));
    const int first = carried + (warp > 0 ? before : 0) + s - v;
    if (e < E) {
      sm.base[e] = first;
      if (offsets) offsets[e] = first;
    }
    carried += __shfl_sync(kAll, c, 31);
    __syncthreads();
  }
  if (offsets && threadIdx.x == 0) offsets[E] = carried;
  return carried;
}

// One block of tokens; ONE: a block of the only cluster, which does the whole
// call, otherwise the first pass of it.
template <int LPT, int EPL, bool FP32, bool ONE>
__global__ void __launch_bounds__(1024, 1) route_choose_kernel(const RouteParams p) {
  __shared__ RouteSmem sm;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int rank = blockIdx.x, ranks = ONE ? gridDim.x : 1;
  const int tokens = ONE ? kOneBlockTokens : p.block_tokens;
  uint16_t *cnt = sm.cnt + warp * p.E;
  ptx::grid_launch_dependents();
  for (int e = lane; e < p.E; e += 32) cnt[e] = 0;
  ptx::grid_dependency_wait();
  const int64_t b0 = int64_t(blockIdx.x) * tokens;
  const int nt = static_cast<int>(max(int64_t(0), min(int64_t(tokens), p.T - b0)));
  // each warp takes a run of tokens, 32 / LPT at a time
  constexpr int SIDE = 32 / LPT;
  const int per = (nt + warps * SIDE - 1) / (warps * SIDE) * SIDE;
  const int t0 = min(warp * per, nt), t1 = min(t0 + per, nt);
  for (int t = t0; t < t1; t += SIDE)
    choose<LPT, EPL, FP32>(p, b0 + t + lane / LPT, b0 + t1, lane, sm.ids + (t + lane / LPT) * p.k);
  __syncwarp();
  walk(sm.ids, t0 * p.k, t1 * p.k, cnt, lane, [](int, unsigned, int) {});
  __syncthreads();
  // the warps' counts of each expert, in order
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
    int run = 0;
    for (int w = 0; w < warps; ++w) {
      const int c = sm.cnt[w * p.E + e];
      sm.cnt[w * p.E + e] = static_cast<uint16_t>(run);
      run += c;
    }
    if (ONE)
      sm.total[e] = sm.base[e] = run;
    else
      p.counts[int64_t(blockIdx.x) * p.E + e] = run;
  }
  if (ONE && ranks > 1) {
    // the cluster's counts, and those of the blocks before this one
    ptx::cluster_sync();
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
      int all = 0, before = 0;
      for (int r = 0; r < ranks; ++r) {
        const int c = static_cast<int>(
            ptx::ld_shared_cluster_u32(ptx::mapa_shared(ptx::smem_u32(&sm.total[e]), r)));
        all += c;
        before += r < rank ? c : 0;
      }
      sm.base[e] = all;
      for (int w = 0; w < warps; ++w) sm.cnt[w * p.E + e] += static_cast<uint16_t>(before);
    }
    // the other blocks have read this one's counts: it may end
    ptx::cluster_sync();
  } else {
    __syncthreads();
  }
  const int routed = ONE ? scan_experts(sm, p.E, rank == 0 ? p.offsets : nullptr) : 0;
  walk(sm.ids, t0 * p.k, t1 * p.k, cnt, lane, [&](int i, unsigned e, int before) {
    const int64_t entry = b0 * p.k + i;
    if (ONE && e != 0xffffu) {
      before += sm.base[e];
      p.rows[before] = static_cast<int32_t>(entry) / p.k;
    }
    p.slots[entry] = e == 0xffffu ? -1 : before;
  });
  if (ONE && rank == 0)
    for (int i = routed + threadIdx.x; i < p.T * p.k; i += blockDim.x) p.rows[i] = -1;
}

// Several blocks, second pass: the block's entries get their places.
__global__ void __launch_bounds__(1024) route_place_kernel(const RouteParams p) {
  __shared__ RouteSmem sm;
  const int b = blockIdx.x;
  ptx::grid_launch_dependents();
  int32_t *mine = sm.total;  // [E] entries of the blocks before this one
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
    sm.base[e] = 0;
    mine[e] = 0;
  }
  ptx::grid_dependency_wait();
  const int64_t b0 = int64_t(b) * p.block_tokens, entries = int64_t(p.T) * p.k;
  const int64_t end = min(b0 + p.block_tokens, int64_t(p.T)) * p.k;
  // the thread's first entry, on its way while the counts are summed
  int64_t i = b0 * p.k + threadIdx.x;
  int e_next = i < end ? __ldg(p.ids + i) : -1, s_next = i < end ? p.slots[i] : 0;
  __syncthreads();
  // Thread (g, e) sums blocks g, g + G, ... of expert e (integer sums in
  // shared memory: their order does not matter).
  const int G = max(1, static_cast<int>(blockDim.x) / p.E);
  for (int e0 = 0; e0 < p.E; e0 += blockDim.x) {
    const int e = e0 + static_cast<int>(threadIdx.x) % p.E;  // E > blockDim.x: e0 + threadIdx.x
    const int g = threadIdx.x / p.E;
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
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) sm.base[e] += mine[e];
  __syncthreads();
  while (i < end) {
    if (e_next >= 0) {
      const int pos = sm.base[e_next] + s_next;
      p.slots[i] = pos;
      p.rows[pos] = static_cast<int32_t>(i) / p.k;  // T * k < 2^31
    }
    i += blockDim.x;
    if (i < end) {
      e_next = __ldg(p.ids + i);
      s_next = p.slots[i];
    }
  }
  for (int64_t n = routed + int64_t(b) * blockDim.x + threadIdx.x; n < entries;
       n += int64_t(p.blocks) * blockDim.x)
    p.rows[n] = -1;
}

cudaError_t launch_pdl(void (*kern)(RouteParams), int grid, int cluster, int threads,
                       const RouteParams &p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

// Tokens per block of the two-launch form: as many blocks as SMs (GB300's 152),
// 32 to 128 tokens each, whole groups of eight (4096 tokens in blocks of 32: 11.3
// us, of 128: 12.7; 1024 tokens 7.8 and 12.0).
int block_tokens(int64_t T) {
  const int64_t n = ((T + 151) / 152 + 7) / 8 * 8;
  return static_cast<int>(std::min<int64_t>(std::max<int64_t>(n, 32), kBlockTokens));
}

// Sizes that the call takes (places and offsets are 32-bit).
bool supported(int64_t T, int64_t E, int64_t k) {
  return E <= kMaxE && k <= kMaxK && T <= ((int64_t(1) << 31) - 1) / k;
}

template <int LPT, int EPL>
cudaError_t launch_route(bool fp32, const RouteParams &p, cudaStream_t s) {
  // warps: as many as there are groups of tokens and counters for
  auto warps = [&](int tokens) { return std::min({32, kCounters / p.E, (tokens + 32 / LPT - 1) / (32 / LPT)}); };
  if (p.T <= kOneTokens) {
    int blocks = 1;  // a power of two
    while (blocks * kOneBlockTokens < p.T) blocks *= 2;
    return launch_pdl(fp32 ? route_choose_kernel<LPT, EPL, true, true>
                           : route_choose_kernel<LPT, EPL, false, true>,
                      blocks, blocks, 32 * warps(std::min(p.T, kOneBlockTokens)), p, s);
  }
  const cudaError_t e = launch_pdl(fp32 ? route_choose_kernel<LPT, EPL, true, false>
                                        : route_choose_kernel<LPT, EPL, false, false>,
                                   p.blocks, 1, 32 * warps(p.block_tokens), p, s);
  return e != cudaSuccess ? e : launch_pdl(route_place_kernel, p.blocks, 1, 1024, p, s);
}

}  // namespace
}  // namespace swiglu

extern "C" uint64_t swiglu_moe_route_workspace_size(int64_t T, int64_t E, int64_t k) {
  using namespace swiglu;
  if (T <= kOneTokens || E < 1 || k < 1 || !supported(T, E, k)) return 0;
  const int n = block_tokens(T);
  return uint64_t((T + n - 1) / n) * E * 4;
}

extern "C" int swiglu_moe_route(const void *logits, int32_t logits_fp32, int32_t renormalize,
                                float scale, int32_t *ids, float *weights, int32_t *offsets,
                                int32_t *rows, int32_t *slots, int64_t T, int64_t E, int64_t k,
                                void *workspace, uint64_t workspace_bytes, void *stream) {
  using namespace swiglu;
  if (T < 0 || E < 1 || k < 1 || k > E || (logits_fp32 != 0 && logits_fp32 != 1) ||
      (renormalize != 0 && renormalize != 1) || !std::isfinite(scale))
    return SWIGLU_ERR_INVALID_ARG;
  if (!supported(T, E, k)) return SWIGLU_ERR_UNSUPPORTED;
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
  p.block_tokens = block_tokens(T);
  p.blocks = int32_t((T + p.block_tokens - 1) / p.block_tokens);
  p.renormalize = renormalize;
  p.scale = scale;
  const bool f = logits_fp32 != 0;
  const int64_t lanes = std::max((E + 7) / 8, k);  // per token
  const cudaError_t e = lanes <= 4    ? launch_route<4, 8>(f, p, s)
                        : lanes <= 8  ? launch_route<8, 8>(f, p, s)
                        : lanes <= 16 ? launch_route<16, 8>(f, p, s)
                        : E <= 256    ? launch_route<32, 8>(f, p, s)
                        : E <= 512    ? launch_route<32, 16>(f, p, s)
                                      : launch_route<32, 32>(f, p, s);
  return e == cudaSuccess ? SWIGLU_OK : SWIGLU_ERR_CUDA;
}
