// k_quant8.cu -- symmetric 8-bit quantisation by rows: a token's activations,
// or an output channel's weights.
//
//     s[r] = max_k |x[r,k]| / 127,   q[r,k] = round(127 x[r,k] / max)
//
// q is the integer nearest to the exact quotient 127 x / max, halves to even.  The
// FP32 product y = x * (127 / max) is off by less than 2^-22 of itself.
//   * BF16: x = X 2^i and max = A 2^j with X, A < 2^8, so a quotient that is no half
//     differs from one by 1 / (2 A 127) or 1 / (127 X) of itself at least, 2^-16;
//     but true halves are common (0.3 % of normal values are max / 2), and y lies to
//     either side of them.  Rounded to 18 bits, y is such a half again, and no
//     other quotient becomes one.
//   * FP32: where y lies within 2^-15 of a half the two sides of 127 |x| <> (m + 1/2)
//     max are compared in FP64, where both products are exact; that is rare.
// Rounding is an addition of 1.5 2^23, whose result holds the code in its low byte:
// conversions run at a quarter of its rate.
//
// One pass: a row stays in the registers of the threads that read it (32 values
// each) up to 32768 values; longer rows are read twice.  A row of up to 1024
// values is one warp's, so that nothing but shuffles joins its maximum.  Bound by
// the copy rate: 65536 rows of 1024 BF16 values 32.9 us, 6.1 TB/s (before the BF16 rule
// above, with the FP64 comparison for both types, 66.6).
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

// Eight values as they are stored.
template <bool FP32>
struct Eight;
template <>
struct Eight<false> {
  uint32_t w[4];
  __device__ __forceinline__ void load(const void *X, int64_t at) {
    const uint4 a = ptx::load(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(X) + at));
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
  }
  __device__ __forceinline__ void clear() { w[0] = w[1] = w[2] = w[3] = 0u; }
  __device__ __forceinline__ float value(int i) const {
    return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
  }
  // The largest magnitude, of it and `top`; NaN where there is one.
  __device__ __forceinline__ float most(float top) const {
    __nv_bfloat162 m = __habs2(pair(0));
#pragma unroll
    for (int i = 1; i < 4; ++i) m = __hmax2_nan(m, __habs2(pair(i)));
    return max_nan(top, max_nan(__low2float(m), __high2float(m)));
  }
  __device__ __forceinline__ __nv_bfloat162 pair(int i) const {
    return *reinterpret_cast<const __nv_bfloat162 *>(&w[i]);
  }
  __device__ static __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
  }
};
template <>
struct Eight<true> {
  float v[8];
  __device__ __forceinline__ void load(const void *X, int64_t at) {
    const float4 *s = reinterpret_cast<const float4 *>(static_cast<const float *>(X) + at);
    const float4 a = ptx::load(s), b = ptx::load(s + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
  }
  __device__ __forceinline__ float value(int i) const { return v[i]; }
  __device__ __forceinline__ float most(float top) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) top = Eight<false>::max_nan(top, fabsf(v[i]));
    return top;
  }
};

// The code of x from its product y with 127 / top, FP32 values.
__device__ __forceinline__ int close_code(float x, float y, float top) {
  if (fabsf(y - rintf(y)) < 0.5f - 0x1p-15f) return static_cast<int>(rintf(y));
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
  Eight<FP32> v[VEC];
  float top = 0.0f;
  if (HELD) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const int64_t k = 8 * int64_t(t + j * TPR);
      v[j].clear();
      if (live && k < p.K) v[j].load(p.X, at + k);
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) top = v[j].most(top);
  } else {
    for (int64_t k = 8 * t; k < p.K; k += 8 * TPR) {
      v[0].load(p.X, at + k);
      top = v[0].most(top);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = Eight<false>::max_nan(top, __shfl_xor_sync(kAll, top, o));
  if (TPR > 32) {
    constexpr int WPR = TPR / 32;  // warps per row
    if (lane == 0) part[warp] = top;
    __syncthreads();
    top = part[warp / WPR * WPR];
#pragma unroll
    for (int i = 1; i < WPR; ++i) top = Eight<false>::max_nan(top, part[warp / WPR * WPR + i]);
  }
  if (!live) return;
  const bool finite = top < CUDART_INF_F;
  if (t == 0) p.scale[row] = finite ? __fdiv_rn(top, 127.0f) : CUDART_NAN_F;
  // a power of two that keeps rows of tiny or huge values away from FP32's ends
  const float up = top < 0x1p-100f ? 0x1p100f : top > 0x1p100f ? 0x1p-20f : 1.0f;
  const float tops = top * up;
  // nothing to scale, or nothing that can be: codes of zero
  const float r = finite && top > 0.0f ? 127.0f / tops : 0.0f;
  auto put = [&](int64_t k, const Eight<FP32> &e) {
    uint32_t w[2] = {0u, 0u};
    if (r != 0.0f) {
      constexpr float RINT = 12582912.0f;  // 1.5 2^23
      float far = 0.0f;                    // from the nearest integer
      uint32_t c[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float y = e.value(i) * up * r;
        if (!FP32) {  // to 18 bits (Veltkamp's splitting)
          const float z = __fmul_rn(y, 65.0f);
          y = __fadd_rn(z, -__fadd_rn(z, -y));
        }
        const float n = __fadd_rn(y, RINT);
        c[i] = __float_as_uint(n);
        if (FP32) far = fmaxf(far, fabsf(y - __fadd_rn(n, -RINT)));
      }
      if (FP32 && far >= 0.5f - 0x1p-15f) {
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
          float x = e.value(0);
#pragma unroll
          for (int j = 1; j < 8; ++j) x = i == j ? e.value(j) : x;
          x *= up;
          const uint32_t k8 = static_cast<uint32_t>(close_code(x, x * r, tops));
#pragma unroll
          for (int j = 0; j < 8; ++j) c[j] = i == j ? k8 : c[j];
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
        w[i] = __byte_perm(__byte_perm(c[4 * i], c[4 * i + 1], 0x0040), __byte_perm(c[4 * i + 2], c[4 * i + 3], 0x0040), 0x5410);
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
      v[0].load(p.X, at + k);
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
