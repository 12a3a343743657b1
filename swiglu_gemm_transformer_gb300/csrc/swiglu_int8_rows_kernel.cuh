// swiglu_int8_rows_kernel.cuh -- products in 8-bit integers for a few rows
// (sm_103a): one token's experts, or one token of a dense layer.
//
//     z[p,n] = sa[p] sw[e,n] sum_k A[p,k] W[e,n,k]         (linear)
//     y[p,n] = SiLU(z1[p,n]) z2[p,n]                       (FUSED)
//
// The sums are exact: dp4a adds four products of 8 bits into 32, and only the
// scaled result is rounded.  Bound by the stream of the weights, each read once
// for up to R rows of its expert: a warp takes NC columns of each matrix, its
// lanes 16 bytes of K each, so that NC (2 NC) loads of 16 bytes are in flight
// per lane; the rows' 16 bytes come from L1, where the block's other warps find
// them too.  Weights pass by L1.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "grouped_units.h"
#include "sm103_ptx.cuh"
#include "tc_common.cuh"

namespace swiglu {

struct Int8RowsParams {
  const int8_t *A, *W1, *W2;
  const float *sa, *s1, *s2;
  const int32_t *offsets;  // [E + 1], or null: one matrix for all rows
  const int32_t *rows;     // [P] or null
  __nv_bfloat16 *Y;        // [P, N]
  int32_t T, P, E, N;
  int64_t K;
  int32_t col_blocks;
};

// 16 bytes of weights, not kept in L1.
__device__ __forceinline__ static uint4 load_weights16(const int8_t *p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ static int dot16(const uint4 &a, const uint4 &b, int c) {
  c = __dp4a(static_cast<int>(a.x), static_cast<int>(b.x), c);
  c = __dp4a(static_cast<int>(a.y), static_cast<int>(b.y), c);
  c = __dp4a(static_cast<int>(a.z), static_cast<int>(b.z), c);
  return __dp4a(static_cast<int>(a.w), static_cast<int>(b.w), c);
}

// The warp's sum as a float.  A lane's part is below 2^31 for K < 2^22, the sum
// of all lanes' only for K < 2^17 (128 * 128 * K).
__device__ __forceinline__ static float warp_sum(int v, bool wide) {
  if (!wide) return static_cast<float>(__reduce_add_sync(0xffffffffu, v));
  long long s = v;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return static_cast<float>(s);
}

constexpr int kRowsMaxExperts = 1024;

// The group bounds, clamped to [0, P] and made not decreasing, and the row tiles
// of R rows before each group: by one warp, to shared memory.
template <int R>
__device__ __forceinline__ static void rows_bounds(const Int8RowsParams &p, int lane, int *off, int *tiles) {
  int top = 0, sum = 0;
  for (int e0 = 0; e0 <= p.E; e0 += 32) {
    const int e = e0 + lane;
    int v = e <= p.E ? min(max(__ldg(p.offsets + e), 0), p.P) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int w = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v = max(v, w);
    }
    v = max(v, top);
    const int prev = __shfl_up_sync(0xffffffffu, v, 1);
    int t = e >= 1 && e <= p.E ? row_tiles<R>(v - (lane == 0 ? top : prev)) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int w = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += w;
    }
    t += sum;
    if (e <= p.E) {
      off[e] = v;
      tiles[e] = t;
    }
    top = __shfl_sync(0xffffffffu, v, 31);
    sum = __shfl_sync(0xffffffffu, t, 31);
  }
}

template <bool FUSED, int R, int NC, int WARPS>
__global__ void __launch_bounds__(32 * WARPS) swiglu_int8_rows_kernel(const __grid_constant__ Int8RowsParams p) {
  constexpr int MATS = FUSED ? 2 : 1;
  __shared__ int off[kRowsMaxExperts + 1], tiles[kRowsMaxExperts + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tile = static_cast<int>(blockIdx.x / p.col_blocks);
  const int col0 = (static_cast<int>(blockIdx.x % p.col_blocks) * WARPS + warp) * NC;
  ptx::grid_launch_dependents();
  ptx::grid_dependency_wait();
  int e = 0, row0, end;
  if (p.offsets) {
    if (warp == 0) rows_bounds<R>(p, lane, off, tiles);
    __syncthreads();
    if (tile >= tiles[p.E]) return;
    int lo = 0, hi = p.E;  // tiles[lo] <= tile < tiles[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (tiles[mid] <= tile) lo = mid; else hi = mid;
    }
    e = lo;
    row0 = off[e] + (tile - tiles[e]) * R;
    end = min(off[e + 1], row0 + R);
  } else {
    row0 = tile * R;
    end = min(p.P, row0 + R);
  }
  if (col0 >= p.N) return;
  const int8_t *a[R];
  int src[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int at = min(row0 + r, end - 1);  // a row past the end repeats the last
    src[r] = p.rows ? __ldg(p.rows + at) : at;
    a[r] = p.A + int64_t(min(max(src[r], 0), p.T - 1)) * p.K + 16 * lane;
  }
  // a column past N repeats the last
  const int8_t *w[MATS][NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int64_t at = (int64_t(e) * p.N + min(col0 + c, p.N - 1)) * p.K + 16 * lane;
    w[0][c] = p.W1 + at;
    if (FUSED) w[MATS - 1][c] = p.W2 + at;
  }
  int acc[MATS][NC][R] = {};
#pragma unroll 2
  for (int64_t k = 16 * lane; k < p.K; k += 512) {
    uint4 x[R], v[MATS][NC];
#pragma unroll
    for (int m = 0; m < MATS; ++m)
#pragma unroll
      for (int c = 0; c < NC; ++c) v[m][c] = load_weights16(w[m][c] + (k - 16 * lane));
#pragma unroll
    for (int r = 0; r < R; ++r) x[r] = __ldg(reinterpret_cast<const uint4 *>(a[r] + (k - 16 * lane)));
#pragma unroll
    for (int m = 0; m < MATS; ++m)
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int r = 0; r < R; ++r) acc[m][c][r] = dot16(v[m][c], x[r], acc[m][c][r]);
  }
  __syncwarp();
  // lane r NC + c finishes row r, column c
  const bool wide = p.K >= (int64_t(1) << 17);
  float g = 0.0f, u = 0.0f;
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const float s = warp_sum(acc[0][c][r], wide);
      g = lane == r * NC + c ? s : g;
      if (FUSED) {
        const float t = warp_sum(acc[MATS - 1][c][r], wide);
        u = lane == r * NC + c ? t : u;
      }
    }
  static_assert(R * NC <= 32, "a lane for each output");
  const int r = lane / NC, row = row0 + r, col = col0 + lane % NC;
  if (r < R && row < end && col < p.N) {
    int from = src[0];
#pragma unroll
    for (int i = 1; i < R; ++i) from = r == i ? src[i] : from;
    float y = 0.0f;  // a row number that names no row of A gives zeros
    if (from >= 0 && from < p.T) {
      const float s = __ldg(p.sa + from);
      const int64_t at = int64_t(e) * p.N + col;
      y = g * s * __ldg(p.s1 + at);
      if (FUSED) y = silu_mul(y, u * s * __ldg(p.s2 + at));
    }
    p.Y[int64_t(row) * p.N + col] = __float2bfloat16_rn(y);
  }
}

}  // namespace swiglu
