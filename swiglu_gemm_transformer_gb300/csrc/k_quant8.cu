// k_quant8.cu -- symmetric 8-bit quantisation by rows: a token's activations,
// or an output channel's weights.
//
//     s[r] = max_k |x[r,k]| / 127,   q[r,k] = round(127 x[r,k] / max)
//
// q is the integer nearest to the exact quotient 127 x / max, halves to even:
// BF16 values meet halves often (max = 254 2^p makes every odd code one).  The
// FP32 product y = x * (127 / max) is off by less than 2^-16, so it decides unless
// it lies within 2^-15 of a half; there the two sides of 127 |x| <> (m + 1/2) max
// are compared in FP64, where both products are exact.
//
// One pass: a row stays in the registers of the threads that read it (32 values
// each) up to 32768 values; longer rows are read twice.  A row of up to 1024
// values is one warp's, so that nothing but shuffles joins its maximum.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "launch.h"
#include "sm103_ptx.cuh"
#include "swiglu.h"

namespace swiglu {
namespace {

struct QuantParams {
  const void *X;
  int8_t *Q;
  float *scale;
  int64_t R, K;
};

constexpr unsigned kAll = 0xffffffffu;

// Eight values.
template <bool FP32>
__device__ __forceinline__ void load8(const void *X, int64_t at, float (&v)[8]) {
  if (FP32) {
    const float4 *s = reinterpret_cast<const float4 *>(static_cast<const float *>(X) + at);
    const float4 a = __ldg(s), b = __ldg(s + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 a = __ldg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(X) + at));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

// A row's code of x: `up` (a power of two) lifts rows of tiny values, r = 127 /
// (top up), top the row's largest magnitude.
__device__ __forceinline__ int code(float x, float up, float r, float top) {
  const float y = x * up * r;
  const float n = rintf(y);
  if (fabsf(y - n) < 0.5f - 0x1p-15f) return static_cast<int>(n);
  const float m = floorf(fabsf(y));  // |y| is next to m + 1/2
  const double d = 127.0 * fabs(double(x)) - (double(m) + 0.5) * double(top);
  const int k = static_cast<int>(m) + (d > 0.0 || (d == 0.0 && (static_cast<int>(m) & 1)) ? 1 : 0);
  return x < 0.0f ? -k : k;
}

// TPR threads per row, a warp or a block; HELD: the row fits their registers.
template <int TPR, bool FP32, bool HELD>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) quant_int8_kernel(const QuantParams p) {
  constexpr int VEC = 4;  // loads of eight values per thread
  constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
  __shared__ float part[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = threadIdx.x % TPR;
  const int64_t row = int64_t(blockIdx.x) * RPB + threadIdx.x / TPR;
  ptx::grid_launch_dependents();
  ptx::grid_dependency_wait();
  const bool live = row < p.R;
  const int64_t at = row * p.K;
  float v[VEC][8];
  float top = 0.0f;
  bool sound = true;  // no NaN (the maximum drops them)
  auto take = [&](const float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      top = fmaxf(top, fabsf(x[i]));
      sound = sound && x[i] == x[i];
    }
  };
  if (HELD) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const int64_t k = 8 * int64_t(t + j * TPR);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = 0.0f;
      if (live && k < p.K) load8<FP32>(p.X, at + k, v[j]);
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) take(v[j]);
  } else {
    for (int64_t k = 8 * t; k < p.K; k += 8 * TPR) {
      load8<FP32>(p.X, at + k, v[0]);
      take(v[0]);
    }
  }
  if (!sound) top = CUDART_INF_F;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
  if (TPR > 32) {
    constexpr int WPR = TPR / 32;  // warps per row
    if (lane == 0) part[warp] = top;
    __syncthreads();
    top = part[warp / WPR * WPR];
#pragma unroll
    for (int i = 1; i < WPR; ++i) top = fmaxf(top, part[warp / WPR * WPR + i]);
  }
  if (!live) return;
  const bool finite = top < CUDART_INF_F;
  const float up = top < 0x1p-100f ? 0x1p100f : 1.0f;
  // nothing to scale, or nothing that can be: codes of zero
  const float r = finite && top > 0.0f ? 127.0f / (top * up) : 0.0f;
  if (t == 0) p.scale[row] = finite ? __fdiv_rn(top, 127.0f) : CUDART_NAN_F;
  auto put = [&](int64_t k, const float (&x)[8]) {
    uint32_t w[2] = {0u, 0u};
    if (r != 0.0f) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        w[i / 4] |= (static_cast<uint32_t>(code(x[i], up, r, top)) & 0xffu) << (8 * (i % 4));
    }
    *reinterpret_cast<uint2 *>(p.Q + at + k) = make_uint2(w[0], w[1]);
  };
  if (HELD) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const int64_t k = 8 * int64_t(t + j * TPR);
      if (k < p.K) put(k, v[j]);
    }
  } else {
    for (int64_t k = 8 * t; k < p.K; k += 8 * TPR) {
      load8<FP32>(p.X, at + k, v[0]);
      put(k, v[0]);
    }
  }
}

template <int TPR, bool HELD>
cudaError_t launch_quant(bool fp32, const QuantParams &p, cudaStream_t s) {
  constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>((p.R + RPB - 1) / RPB));
  cfg.blockDim = dim3(TPR * RPB);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fp32 ? quant_int8_kernel<TPR, true, HELD> : quant_int8_kernel<TPR, false, HELD>,
                            p);
}

}  // namespace
}  // namespace swiglu

extern "C" int swiglu_quant_int8(const void *X, int32_t x_fp32, void *Q, float *scale, int64_t R,
                                 int64_t K, void *stream) {
  using namespace swiglu;
  if (R < 0 || K < 0 || (x_fp32 != 0 && x_fp32 != 1)) return SWIGLU_ERR_INVALID_ARG;
  if (R >= int64_t(1) << 31 || K >= int64_t(1) << 31) return SWIGLU_ERR_UNSUPPORTED;
  if (R == 0) return SWIGLU_OK;
  if (!scale || (K > 0 && (!X || !Q))) return SWIGLU_ERR_INVALID_ARG;
  if (!ptr_aligned(scale, 4) || (K > 0 && (!ptr_aligned(X, 16) || !ptr_aligned(Q, 8))) || K % 8 != 0)
    return SWIGLU_ERR_MISALIGNED;
  const uint64_t xn = uint64_t(R) * K * (x_fp32 ? 4 : 2), qn = uint64_t(R) * K, sn = uint64_t(R) * 4;
  if (ranges_overlap(Q, qn, X, xn) || ranges_overlap(scale, sn, X, xn) || ranges_overlap(scale, sn, Q, qn))
    return SWIGLU_ERR_INVALID_ARG;
  uint32_t *err = nullptr;
  int sms = 0;
  uint64_t timeout_ns = 0, gen = 0;
  const int rc = device_info(&err, &sms, &timeout_ns, &gen);
  if (rc != SWIGLU_OK) return rc;
  const QuantParams p = {X, static_cast<int8_t *>(Q), scale, R, K};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool f = x_fp32 != 0;
  const cudaError_t e = K <= 1024    ? launch_quant<32, true>(f, p, s)
                        : K <= 4096  ? launch_quant<128, true>(f, p, s)
                        : K <= 8192  ? launch_quant<256, true>(f, p, s)
                        : K <= 32768 ? launch_quant<1024, true>(f, p, s)
                                     : launch_quant<1024, false>(f, p, s);
  return e == cudaSuccess ? SWIGLU_OK : SWIGLU_ERR_CUDA;
}
