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
// once, R' and H written once.  One block per row holds the row in registers,
// eight columns per thread and vector, so the two sums (each a block
// reduction, the second over values that depend on the first) cost no second
// pass; the loads of R, the gate and the norms' weights are issued before the
// first reduction.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "launch.h"
#include "sm103_ptx.cuh"
#include "swiglu.h"

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
__global__ void __launch_bounds__(THREADS) residual_norm_kernel(const NormParams p) {
  __shared__ float red[2][32];
  ptx::grid_launch_dependents();
  ptx::grid_dependency_wait();
  const int64_t t = blockIdx.x;
  const int nv = p.D / 8;
  float z[VPT][8];
  uint4 rb[VPT], gb[VPT];
  float4 rf[R32 ? VPT : 1][2];
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
    if (p.gate) gb[i] = __ldg(reinterpret_cast<const uint4 *>(p.gate + t * p.gate_stride) + v);
  }
  const uint4 *Z = reinterpret_cast<const uint4 *>(p.Z);
  if (p.slots == nullptr) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * THREADS;
      if (v < nv) bf16x8(__ldg(Z + t * nv + v), z[i]);
    }
  } else {
#pragma unroll 8
    for (int j = 0; j < p.k; ++j) {
      const int s = __ldg(p.slots + t * p.k + j);
      if (s < 0 || s >= p.P) continue;
      const float w = __ldg(p.weights + t * p.k + j);
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = threadIdx.x + i * THREADS;
        if (v >= nv) continue;
        float f[8];
        bf16x8(__ldg(Z + int64_t(s) * nv + v), f);
#pragma unroll
        for (int c = 0; c < 8; ++c) z[i][c] = fmaf(w, f[c], z[i][c]);
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
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + i * THREADS;
    if (v >= nv) continue;
    float f[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) z[i][c] *= scale;
    if (p.gamma_post) {
      bf16x8(__ldg(reinterpret_cast<const uint4 *>(p.gamma_post) + v), f);
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
  scale = inv_root(block_sum<THREADS>(ss, red[1]), inv_d, p.eps);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + i * THREADS;
    if (v >= nv) continue;
    float f[8];
    if (p.gamma_pre) {
      bf16x8(__ldg(reinterpret_cast<const uint4 *>(p.gamma_pre) + v), f);
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
  const cudaError_t e = nv <= 32     ? launch_norm<32, 1>(r32, p, s)
                        : nv <= 128  ? launch_norm<128, 1>(r32, p, s)
                        : nv <= 256  ? launch_norm<256, 1>(r32, p, s)
                        : nv <= 512  ? launch_norm<512, 1>(r32, p, s)
                        : nv <= 1024 ? launch_norm<512, 2>(r32, p, s)
                        : nv <= 2048 ? launch_norm<1024, 2>(r32, p, s)
                                     : launch_norm<1024, 4>(r32, p, s);
  return e == cudaSuccess ? SWIGLU_OK : SWIGLU_ERR_CUDA;
}
