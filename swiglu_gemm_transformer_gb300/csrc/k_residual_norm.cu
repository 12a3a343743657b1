// k_residual_norm.cu -- the end of a block: the join of the experts' rows,
// the norm after the block, its gate and residual, and the norm before the
// next block, in one pass over the rows.
//
//     z  = Z[t], or sum_j weights[t,j] Z[slots[t,j]]
//     n  = z * gamma_post / sqrt(mean z^2 + eps)      (or z without that norm)
//     R' = s R + g (.) n
//     H  = R' * gamma_pre / sqrt(mean R'^2 + eps)
//
// All of it is FP32; R' (in R's type) and H (BF16) are rounded once, and H is
// made from the unrounded R'.  Bound by memory: Z, R and the gate are read
// once, R' and H written once.  A block holds a row in registers, eight columns
// per thread and vector, so the two sums (each a block reduction, the second
// over values that depend on the first) cost no second pass.
//
// Two kernels:
//   * few rows (up to kDirectRows per SM): one block per row, loading straight
//     to registers, all loads issued before the first reduction;
//   * more rows: persistent blocks; a warp of its own copies the rows ahead
//     into a ring in shared memory with bulk copies (one per expert's row, one
//     for R, one for the gate), so that memory stays busy through the
//     reductions, and the norms' weights stay in registers from row to row.
//     Its outputs are stored evict-first (8191 rows x 8192, FP32 residual and a
//     gate per row: 156.5 -> 151.2 us; now 156.6; 8192 rows x 2048, 8 joined: 59.9).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "launch.h"
#include "sm103_ptx.cuh"
#include "swiglu.h"
#include "tc_common.cuh"

namespace swiglu {
namespace {

struct NormParams {
  const __nv_bfloat16 *Z;
  const int32_t *slots;    // [T, k] or null
  const float *weights;    // [T, k] or null (with slots)
  const void *R;           // [T, D] BF16 or FP32
  const __nv_bfloat16 *gamma_post, *gate, *gamma_pre;  // or null
  int64_t gate_stride;     // elements between the rows of the gate; 0 = one row for all
  void *Rout;
  __nv_bfloat16 *H;        // or null
  int32_t T, P, k, D;
  int32_t post_norm;
  float residual_scale, eps;
};

__device__ __forceinline__ void bf16x8(const uint4 v, float f[8]) {
  f[0] = __uint_as_float(v.x << 16);
  f[1] = __uint_as_float(v.x & 0xFFFF0000u);
  f[2] = __uint_as_float(v.y << 16);
  f[3] = __uint_as_float(v.y & 0xFFFF0000u);
  f[4] = __uint_as_float(v.z << 16);
  f[5] = __uint_as_float(v.z & 0xFFFF0000u);
  f[6] = __uint_as_float(v.w << 16);
  f[7] = __uint_as_float(v.w & 0xFFFF0000u);
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t *>(&v);
}

// Sum over the block; every thread gets it.  `red` has one slot per warp.
template <int THREADS>
__device__ __forceinline__ float block_sum(float v, float *red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (THREADS == 32) return v;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  constexpr int W = THREADS / 32;
  float s = (threadIdx.x & 31) < W ? red[threadIdx.x & 31] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// 1/sqrt(mean + eps); 0 where that is 1/0 (a row of zeros with eps = 0).
__device__ __forceinline__ float inv_root(float sum, float inv_d, float eps) {
  const float d = fmaf(sum, inv_d, eps);
  return d == 0.0f ? 0.0f : 1.0f / sqrtf(d);
}

template <int THREADS, int VPT, bool R32>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) residual_norm_kernel(const NormParams p) {
  __shared__ float red[2][32];
  ptx::grid_launch_dependents();
  ptx::grid_dependency_wait();
  const int64_t t = blockIdx.x;
  const int nv = p.D / 8;
  float z[VPT][8];
  uint4 rb[VPT], gb[VPT];
  float4 rf[R32 ? VPT : 1][2];
  // The norms' weights: loaded at once where registers suffice, else a vector ahead of
  // its use (loads do not pass the stores before them).
  constexpr bool EARLY = VPT == 1;
  uint4 gpost[VPT], gpre[VPT];
  auto load_gamma = [&](uint4 (&g)[VPT], const __nv_bfloat16 *gamma, int i) {
    const int v = threadIdx.x + i * THREADS;
    if (i < VPT && gamma && v < nv) g[i] = ptx::load(reinterpret_cast<const uint4 *>(gamma) + v);
  };
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + i * THREADS;
#pragma unroll
    for (int c = 0; c < 8; ++c) z[i][c] = 0.0f;
    if (v >= nv) continue;
    if (R32) {
      const float4 *r = static_cast<const float4 *>(p.R) + t * (p.D / 4) + 2 * v;
      rf[i][0] = r[0];
      rf[i][1] = r[1];
    } else {
      rb[i] = static_cast<const uint4 *>(p.R)[t * nv + v];
    }
    if (p.gate) gb[i] = ptx::load(reinterpret_cast<const uint4 *>(p.gate + t * p.gate_stride) + v);
    if (EARLY) load_gamma(gpost, p.gamma_post, i);
    if (EARLY) load_gamma(gpre, p.gamma_pre, i);
  }
  const uint4 *Z = reinterpret_cast<const uint4 *>(p.Z);
  if (p.slots == nullptr) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * THREADS;
      if (v < nv) bf16x8(ptx::load(Z + t * nv + v), z[i]);
    }
  } else {
    // CH choices at a time, all their loads issued before the first use; a
    // slot that names nothing is loaded as zeros
    constexpr int CH = VPT <= 2 ? 4 : 2;
    for (int j0 = 0; j0 < p.k; j0 += CH) {
      int slot[CH];
      float w[CH];
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        slot[j] = j0 + j < p.k ? ptx::load(p.slots + t * p.k + j0 + j) : -1;
        w[j] = j0 + j < p.k ? ptx::load(p.weights + t * p.k + j0 + j) : 0.0f;
      }
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        if (slot[j] >= p.P) slot[j] = -1;
        if (slot[j] < 0) w[j] = 0.0f;
      }
      uint4 x[CH][VPT];
#pragma unroll
      for (int j = 0; j < CH; ++j)
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          const int v = threadIdx.x + i * THREADS;
          x[j][i] = slot[j] >= 0 && v < nv ? ptx::load(Z + int64_t(slot[j]) * nv + v)
                                           : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
      for (int j = 0; j < CH; ++j)
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          float f[8];
          bf16x8(x[j][i], f);
#pragma unroll
          for (int c = 0; c < 8; ++c) z[i][c] = fmaf(w[j], f[c], z[i][c]);
        }
    }
  }
  const float inv_d = 1.0f / p.D;
  float scale = 1.0f;
  if (p.post_norm) {
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int c = 0; c < 8; ++c) ss = fmaf(z[i][c], z[i][c], ss);
    scale = inv_root(block_sum<THREADS>(ss, red[0]), inv_d, p.eps);
  }
  float ss = 0.0f;
  if (!EARLY) load_gamma(gpost, p.gamma_post, 0);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + i * THREADS;
    if (v >= nv) continue;
    if (!EARLY) load_gamma(gpost, p.gamma_post, i + 1);
    float f[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) z[i][c] *= scale;
    if (p.gamma_post) {
      bf16x8(gpost[i], f);
#pragma unroll
      for (int c = 0; c < 8; ++c) z[i][c] *= f[c];
    }
    if (p.gate) {
      bf16x8(gb[i], f);
#pragma unroll
      for (int c = 0; c < 8; ++c) z[i][c] *= f[c];
    }
    if (R32) {
      f[0] = rf[i][0].x, f[1] = rf[i][0].y, f[2] = rf[i][0].z, f[3] = rf[i][0].w;
      f[4] = rf[i][1].x, f[5] = rf[i][1].y, f[6] = rf[i][1].z, f[7] = rf[i][1].w;
    } else {
      bf16x8(rb[i], f);
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      z[i][c] = fmaf(p.residual_scale, f[c], z[i][c]);
      ss = fmaf(z[i][c], z[i][c], ss);
    }
    if (R32) {
      float4 *o = static_cast<float4 *>(p.Rout) + t * (p.D / 4) + 2 * v;
      o[0] = make_float4(z[i][0], z[i][1], z[i][2], z[i][3]);
      o[1] = make_float4(z[i][4], z[i][5], z[i][6], z[i][7]);
    } else {
      static_cast<uint4 *>(p.Rout)[t * nv + v] =
          make_uint4(pack2(z[i][0], z[i][1]), pack2(z[i][2], z[i][3]), pack2(z[i][4], z[i][5]),
                     pack2(z[i][6], z[i][7]));
    }
  }
  if (p.H == nullptr) return;
  if (!EARLY) load_gamma(gpre, p.gamma_pre, 0);
  scale = inv_root(block_sum<THREADS>(ss, red[1]), inv_d, p.eps);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + i * THREADS;
    if (v >= nv) continue;
    if (!EARLY) load_gamma(gpre, p.gamma_pre, i + 1);
    float f[8];
    if (p.gamma_pre) {
      bf16x8(gpre[i], f);
#pragma unroll
      for (int c = 0; c < 8; ++c) f[c] *= z[i][c] * scale;
    } else {
#pragma unroll
      for (int c = 0; c < 8; ++c) f[c] = z[i][c] * scale;
    }
    reinterpret_cast<uint4 *>(p.H)[t * nv + v] =
        make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
  }
}

// Eight columns of R as floats.
template <bool R32>
__device__ __forceinline__ void residual8(const uint8_t *row, int v, float f[8]) {
  if (R32) {
    const float4 a = reinterpret_cast<const float4 *>(row)[2 * v];
    const float4 b = reinterpret_cast<const float4 *>(row)[2 * v + 1];
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  } else {
    bf16x8(reinterpret_cast<const uint4 *>(row)[v], f);
  }
}

constexpr int kRingMaxK = 32;    // choices per token: one lane of the copying warp each
constexpr int kRingMaxStages = 8;

// Ring of a persistent block: per stage kr rows of Z (k, or 1 without slots),
// R's row and, where the gate has rows, the gate's; then, for every stage, the
// weights and a mask of the slots that name a row; the barriers.
struct RingLayout {
  uint32_t z_bytes, r_bytes, g_bytes, stage_bytes, side_off, bar_off, total;
  int stages;
};

__host__ __device__ inline RingLayout ring_layout(int D, int kr, bool r32, bool gate_rows, int stages) {
  RingLayout l;
  l.z_bytes = uint32_t(D) * 2;
  l.r_bytes = uint32_t(D) * (r32 ? 4 : 2);
  l.g_bytes = gate_rows ? uint32_t(D) * 2 : 0;
  l.stage_bytes = l.z_bytes * kr + l.r_bytes + l.g_bytes;
  l.stages = stages;
  l.side_off = l.stage_bytes * stages;
  l.bar_off = l.side_off + stages * (kRingMaxK + 4) * 4;
  l.total = l.bar_off + stages * 16 + 16;
  return l;
}

// Most blocks per SM: what their registers leave room for.
constexpr int ring_most_blocks(int threads, int vpt) {
  return threads == 32 ? 16 : threads == 64 ? 8 : threads == 128 ? (vpt == 1 ? 6 : 4) : threads == 256 ? 2 : 1;
}

template <int THREADS, int VPT, bool R32>
__global__ void __launch_bounds__(THREADS + 32, ring_most_blocks(THREADS, VPT))
    residual_norm_ring_kernel(const NormParams p, const RingLayout l, uint32_t *err,
                              uint64_t timeout_ns) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float red[2][2][32];  // [sum][row parity]: one barrier a sum is enough
  constexpr int WARPS = THREADS / 32;
  const uint32_t bars = ptx::smem_u32(smem + l.bar_off);
  auto full = [&](uint32_t s) { return bars + 16u * s; };
  auto empty = [&](uint32_t s) { return bars + 16u * s + 8u; };
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + l.bar_off + 16 * l.stages);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nv = p.D / 8, kr = p.slots ? p.k : 1;
  if (threadIdx.x == 0) {
    for (int s = 0; s < l.stages; ++s) {
      ptx::mbar_init(full(s), 1);
      ptx::mbar_init(empty(s), WARPS);
    }
    *abort_flag = 0;
    ptx::fence_barrier_init();
  }
  __syncthreads();
  ptx::grid_launch_dependents();
  ptx::grid_dependency_wait();
  uint32_t stage = 0, phase = 0;

  if (warp == WARPS) {
    // ------------------------------------------------------------ copies
    // lane j: row j of Z and its weight; the last two lanes: R and the gate
    auto choice = [&](int64_t t, int &slot, float &w) {
      slot = -1;
      w = 0.0f;
      if (t >= p.T || lane >= kr) return;
      slot = p.slots ? ptx::load(p.slots + t * p.k + lane) : static_cast<int>(t);
      if (slot < 0 || slot >= p.P) slot = -1;
      if (p.slots && slot >= 0) w = ptx::load(p.weights + t * p.k + lane);
    };
    int slot;
    float w;
    choice(blockIdx.x, slot, w);
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
      bool ok = true;
      if (lane == 0) ok = wait_bar(empty(stage), phase ^ 1u, timeout_ns, abort_flag, err, WAIT_PRODUCER_EMPTY);
      if (!__shfl_sync(0xffffffffu, ok, 0)) {
        spin_ns(100000);  // aborted: copies already in flight land
        break;
      }
      // lane 0 saw that the rows' warps have read the stage: now every lane may
      // write it (shuffles and ballots order no memory)
      __syncwarp();
      uint8_t *side = smem + l.side_off + stage * (kRingMaxK + 4) * 4;
      reinterpret_cast<float *>(side)[lane] = w;
      const uint32_t mask = __ballot_sync(0xffffffffu, slot >= 0);
      const uint32_t dst = ptx::smem_u32(smem) + stage * l.stage_bytes;
      // the lanes' weights are written before lane 0's arrival hands them to the
      // rows' warps, and the bytes are expected before the copies start
      __syncwarp();
      if (lane == 0) {
        reinterpret_cast<uint32_t *>(side)[kRingMaxK] = mask;
        ptx::mbar_arrive_expect_tx(full(stage), l.z_bytes * __popc(mask) + l.r_bytes + l.g_bytes);
      }
      __syncwarp();
      if (slot >= 0)
        ptx::bulk_load(dst + lane * l.z_bytes, p.Z + int64_t(slot) * p.D, l.z_bytes, full(stage));
      if (lane == 30)
        ptx::bulk_load(dst + kr * l.z_bytes, static_cast<const uint8_t *>(p.R) + t * l.r_bytes,
                       l.r_bytes, full(stage));
      if (lane == 31 && l.g_bytes)
        ptx::bulk_load(dst + kr * l.z_bytes + l.r_bytes, p.gate + t * p.gate_stride, l.g_bytes,
                       full(stage));
      choice(t + gridDim.x, slot, w);  // of the next row, in flight through the wait
      if (++stage == uint32_t(l.stages)) {
        stage = 0;
        phase ^= 1u;
      }
    }
    return;
  }

  // -------------------------------------------------------------- rows
  auto group_sum = [&](float v, float *slots) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (WARPS == 1) return v;
    if (lane == 0) slots[warp] = v;
    asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
    float s = lane < WARPS ? slots[lane] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
  };
  // The norms' weights and a gate of one row stay in registers where these
  // suffice; longer rows read them again (from L1 or L2) for every row.
  constexpr bool HOLD = VPT <= 2;
  // A gate of one row and that of the row at hand share registers, but for FP32 rows of
  // up to 4096 (8191 rows of 4096 76 us with registers of their own, 88 without).
  constexpr bool SHARE = !R32 || THREADS > 256;
  uint4 gpost[VPT], gpre[VPT], gvec[VPT];
  const bool gate_vec = p.gate && !l.g_bytes;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + i * THREADS;
    if (!HOLD || v >= nv) continue;
    if (p.gamma_post) gpost[i] = ptx::load(reinterpret_cast<const uint4 *>(p.gamma_post) + v);
    if (p.gamma_pre) gpre[i] = ptx::load(reinterpret_cast<const uint4 *>(p.gamma_pre) + v);
    if (gate_vec) gvec[i] = ptx::load(reinterpret_cast<const uint4 *>(p.gate) + v);
  }
  const float inv_d = 1.0f / p.D;
  int parity = 0;
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, parity ^= 1) {
    // all warps go on or none: a wait that gives up sets the block's flag, and
    // the rows' barrier that follows is reached either way
    const bool ok = wait_bar(full(stage), phase, timeout_ns, abort_flag, err, WAIT_MMA_FULL);
    const uint8_t *src = smem + stage * l.stage_bytes;
    const uint8_t *side = smem + l.side_off + stage * (kRingMaxK + 4) * 4;
    const uint32_t mask = ok ? reinterpret_cast<const uint32_t *>(side)[kRingMaxK] : 0u;
    float z[VPT][8], f[8];
    float ss = 0.0f;
    float r[VPT][8];
    uint4 own[VPT];
    auto &gb = SHARE ? gvec : own;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * THREADS;
#pragma unroll
      for (int c = 0; c < 8; ++c) z[i][c] = 0.0f;
      if (v >= nv) continue;
      if (p.slots == nullptr) {
        if (mask) bf16x8(reinterpret_cast<const uint4 *>(src)[v], z[i]);
      } else {
        for (uint32_t m = mask; m; m &= m - 1u) {
          const int j = __ffs(m) - 1;
          const float w = reinterpret_cast<const float *>(side)[j];
          bf16x8(reinterpret_cast<const uint4 *>(src + j * l.z_bytes)[v], f);
#pragma unroll
          for (int c = 0; c < 8; ++c) z[i][c] = fmaf(w, f[c], z[i][c]);
        }
      }
#pragma unroll
      for (int c = 0; c < 8; ++c) ss = fmaf(z[i][c], z[i][c], ss);
      residual8<R32>(src + kr * l.z_bytes, v, r[i]);
      if (l.g_bytes) gb[i] = reinterpret_cast<const uint4 *>(src + kr * l.z_bytes + l.r_bytes)[v];
    }
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(empty(stage));  // the stage is in registers
    if (++stage == uint32_t(l.stages)) {
      stage = 0;
      phase ^= 1u;
    }
    float scale = 1.0f;
    if (p.post_norm) scale = inv_root(group_sum(ss, red[0][parity]), inv_d, p.eps);
    ss = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * THREADS;
      if (v >= nv) continue;
#pragma unroll
      for (int c = 0; c < 8; ++c) z[i][c] *= scale;
      if (p.gamma_post) {
        bf16x8(HOLD ? gpost[i] : ptx::load(reinterpret_cast<const uint4 *>(p.gamma_post) + v), f);
#pragma unroll
        for (int c = 0; c < 8; ++c) z[i][c] *= f[c];
      }
      if (p.gate) {
        bf16x8(!gate_vec ? gb[i] : HOLD ? gvec[i] : ptx::load(reinterpret_cast<const uint4 *>(p.gate) + v), f);
#pragma unroll
        for (int c = 0; c < 8; ++c) z[i][c] *= f[c];
      }
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        z[i][c] = fmaf(p.residual_scale, r[i][c], z[i][c]);
        ss = fmaf(z[i][c], z[i][c], ss);
      }
      if (!ok) continue;
      if (R32) {
        float4 *o = static_cast<float4 *>(p.Rout) + t * (p.D / 4) + 2 * v;
        __stcs(o, make_float4(z[i][0], z[i][1], z[i][2], z[i][3]));
        __stcs(o + 1, make_float4(z[i][4], z[i][5], z[i][6], z[i][7]));
      } else {
        __stcs(static_cast<uint4 *>(p.Rout) + t * nv + v,
            make_uint4(pack2(z[i][0], z[i][1]), pack2(z[i][2], z[i][3]), pack2(z[i][4], z[i][5]),
                       pack2(z[i][6], z[i][7])));
      }
    }
    if (p.H == nullptr) continue;
    scale = inv_root(group_sum(ss, red[1][parity]), inv_d, p.eps);
    if (!ok) continue;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * THREADS;
      if (v >= nv) continue;
      if (p.gamma_pre) {
        bf16x8(HOLD ? gpre[i] : ptx::load(reinterpret_cast<const uint4 *>(p.gamma_pre) + v), f);
#pragma unroll
        for (int c = 0; c < 8; ++c) f[c] *= z[i][c] * scale;
      } else {
#pragma unroll
        for (int c = 0; c < 8; ++c) f[c] = z[i][c] * scale;
      }
      __stcs(reinterpret_cast<uint4 *>(p.H) + t * nv + v,
          make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7])));
    }
  }
}

template <int THREADS, int VPT>
cudaError_t launch_ring(bool r32, const NormParams &p, int per_sm, int stages, int sms,
                        uint32_t *err, uint64_t timeout_ns, uint64_t ctx_gen, cudaStream_t s) {
  static PerDeviceOnce once;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (once.needed(dev, ctx_gen)) {
    e = cudaFuncSetAttribute(residual_norm_ring_kernel<THREADS, VPT, true>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, 224 * 1024);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(residual_norm_ring_kernel<THREADS, VPT, false>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, 224 * 1024);
    if (e != cudaSuccess) return e;
    once.done(dev, ctx_gen);
  }
  const RingLayout l = ring_layout(p.D, p.slots ? p.k : 1, r32, p.gate && p.gate_stride, stages);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  const int64_t grid = int64_t(per_sm) * sms;
  cfg.gridDim = dim3(static_cast<unsigned>(grid < p.T ? grid : p.T));
  cfg.blockDim = dim3(THREADS + 32);
  cfg.dynamicSmemBytes = l.total;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, r32 ? residual_norm_ring_kernel<THREADS, VPT, true>
                                      : residual_norm_ring_kernel<THREADS, VPT, false>,
                            p, l, err, timeout_ns);
}

template <int THREADS, int VPT>
cudaError_t launch_norm(bool r32, const NormParams &p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(p.T));
  cfg.blockDim = dim3(THREADS);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, r32 ? residual_norm_kernel<THREADS, VPT, true>
                                      : residual_norm_kernel<THREADS, VPT, false>, p);
}

constexpr int64_t kMaxCols = 32768;  // 1024 threads x 4 vectors of 8
constexpr int64_t kDirectRows = 4;   // rows per SM up to which blocks load directly

// Blocks per SM and stages of the ring kernel, or 0 where it does not apply:
// as many blocks as leave each two stages (their reductions hide each
// other's), then as many stages as fit.
int ring_blocks(int D, int kr, bool r32, bool gate_rows, int most, int *stages) {
  if (kr > kRingMaxK - 2) return 0;
  const int budget = 224 * 1024;
  for (int c = most; c >= 1; --c) {
    const int mine = budget / c - 1536;  // each block also takes 1 KB of the SM, and `red`
    int st = kRingMaxStages;
    while (st >= 2 && int64_t(ring_layout(D, kr, r32, gate_rows, st).total) > mine) --st;
    if (st >= 2) {
      *stages = st;
      return c;
    }
  }
  return 0;
}

}  // namespace
}  // namespace swiglu

extern "C" int swiglu_residual_norm(const void *Z, const int32_t *slots, const float *weights,
                                    const void *R, int32_t r_fp32, int32_t post_norm,
                                    const void *gamma_post, const void *gate, int64_t gate_stride,
                                    float residual_scale, const void *gamma_pre, float eps,
                                    void *Rout, void *H, int64_t T, int64_t P, int64_t k, int64_t D,
                                    void *stream) {
  using namespace swiglu;
  if (T < 0 || P < 0 || k < 0 || D < 0 || gate_stride < 0 || (r_fp32 != 0 && r_fp32 != 1) ||
      (post_norm != 0 && post_norm != 1) || !(eps >= 0.0f) || !std::isfinite(eps) ||
      !std::isfinite(residual_scale))
    return SWIGLU_ERR_INVALID_ARG;
  const int64_t limit = (int64_t(1) << 31) - 1;
  if (T > limit || P > limit || k > limit || D > kMaxCols) return SWIGLU_ERR_UNSUPPORTED;
  if (T == 0 || D == 0) return SWIGLU_OK;
  if (!R || !Rout || (P > 0 && !Z) || (slots && k > 0 && !weights) || (!slots && P != T))
    return SWIGLU_ERR_INVALID_ARG;
  if (gamma_post && !post_norm) return SWIGLU_ERR_INVALID_ARG;
  if (gate && gate_stride != 0 && gate_stride < D) return SWIGLU_ERR_INVALID_ARG;
  if (D % 8 != 0 || (gate && gate_stride % 8 != 0)) return SWIGLU_ERR_MISALIGNED;
  if (!ptr_aligned(Z, 16) || !ptr_aligned(R, 16) || !ptr_aligned(gamma_post, 16) ||
      !ptr_aligned(gate, 16) || !ptr_aligned(gamma_pre, 16) || !ptr_aligned(Rout, 16) ||
      !ptr_aligned(H, 16) || !ptr_aligned(slots, 4) || !ptr_aligned(weights, 4))
    return SWIGLU_ERR_MISALIGNED;
  // R' may be R itself (every element is read before it is written, by the
  // same thread); nothing else may overlap an output
  const uint64_t r_bytes = uint64_t(T) * D * (r_fp32 ? 4 : 2), h_bytes = uint64_t(T) * D * 2;
  const void *in[7] = {Z, slots, weights, gamma_post, gate, gamma_pre, R};
  const uint64_t in_len[7] = {uint64_t(P) * D * 2, uint64_t(T) * k * 4, uint64_t(T) * k * 4,
                              uint64_t(D) * 2, (uint64_t(T - 1) * gate_stride + D) * 2,
                              uint64_t(D) * 2, r_bytes};
  for (int i = 0; i < 7; ++i) {
    if (ranges_overlap(H, h_bytes, in[i], in_len[i])) return SWIGLU_ERR_INVALID_ARG;
    if (!(i == 6 && R == Rout) && ranges_overlap(Rout, r_bytes, in[i], in_len[i]))
      return SWIGLU_ERR_INVALID_ARG;
  }
  if (ranges_overlap(H, h_bytes, Rout, r_bytes)) return SWIGLU_ERR_INVALID_ARG;
  uint32_t *err = nullptr;
  int sms = 0;
  uint64_t timeout_ns = 0, gen = 0;
  int rc = device_info(&err, &sms, &timeout_ns, &gen);
  if (rc != SWIGLU_OK) return rc;
  NormParams p;
  p.Z = static_cast<const __nv_bfloat16 *>(Z);
  p.slots = slots;
  p.weights = weights;
  p.R = R;
  p.gamma_post = static_cast<const __nv_bfloat16 *>(gamma_post);
  p.gate = static_cast<const __nv_bfloat16 *>(gate);
  p.gamma_pre = static_cast<const __nv_bfloat16 *>(gamma_pre);
  p.gate_stride = gate_stride;
  p.Rout = Rout;
  p.H = static_cast<__nv_bfloat16 *>(H);
  p.T = int32_t(T);
  p.P = int32_t(P);
  p.k = int32_t(k);
  p.D = int32_t(D);
  p.post_norm = post_norm;
  p.residual_scale = residual_scale;
  p.eps = eps;
  const bool r32 = r_fp32 != 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t nv = D / 8;
  const int ring_threads = nv <= 32 ? 32 : nv <= 64 ? 64 : nv <= 256 ? 128 : nv <= 512 ? 256 : 512;
  const int ring_vpt = nv <= 128 ? 1 : nv <= 1024 ? 2 : 4;
  int stages = 0;
  const int per_sm = nv <= 2048 && T > kDirectRows * sms
                         ? ring_blocks(p.D, slots ? p.k : 1, r32, gate && gate_stride,
                                       ring_most_blocks(ring_threads, ring_vpt), &stages)
                         : 0;
  if (per_sm > 0 && !(slots && k == 0)) {
    auto go = [&](auto launch) { return launch(r32, p, per_sm, stages, sms, err, timeout_ns, gen, s); };
    const cudaError_t e = nv <= 32     ? go(launch_ring<32, 1>)
                          : nv <= 64   ? go(launch_ring<64, 1>)
                          : nv <= 128  ? go(launch_ring<128, 1>)
                          : nv <= 256  ? go(launch_ring<128, 2>)
                          : nv <= 512  ? go(launch_ring<256, 2>)
                          : nv <= 1024 ? go(launch_ring<512, 2>)
                                       : go(launch_ring<512, 4>);
    return e == cudaSuccess ? SWIGLU_OK : SWIGLU_ERR_CUDA;
  }
  const cudaError_t e = nv <= 32     ? launch_norm<32, 1>(r32, p, s)
                        : nv <= 128  ? launch_norm<128, 1>(r32, p, s)
                        : nv <= 256  ? launch_norm<256, 1>(r32, p, s)
                        : nv <= 512  ? launch_norm<512, 1>(r32, p, s)
                        : nv <= 1024 ? launch_norm<512, 2>(r32, p, s)
                        : nv <= 2048 ? launch_norm<1024, 2>(r32, p, s)
                                     : launch_norm<1024, 4>(r32, p, s);
  return e == cudaSuccess ? SWIGLU_OK : SWIGLU_ERR_CUDA;
}
