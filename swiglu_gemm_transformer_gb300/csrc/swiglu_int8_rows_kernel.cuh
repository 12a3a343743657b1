// swiglu_int8_rows_kernel.cuh -- products in 8-bit integers for a few rows
// (sm_103a): a few tokens' experts, or a few rows of a dense layer.
//
//     z[p,n] = sa[p] sw[e,n] sum_k A[p,k] W[e,n,k]         (linear)
//     y[p,n] = SiLU(z1[p,n]) z2[p,n]                       (FUSED)
//
// Both kernels are bound by the stream of the weights, which goes from memory
// straight to registers, 16 bytes of a column a lane, past L1.  Sums of products
// are 32-bit integers, exact whatever their order.
//   * swiglu_int8_token_kernel, one row: a warp takes NC columns of each matrix,
//     its lanes 512 bytes of K a turn, and dp4a adds four products at once.
//   * swiglu_int8_rows_kernel, up to 8 rows: a block takes 16 columns of each
//     matrix, its warps K in turns of 128, by the integer MMA of a warp (m16n8k32):
//     a tenth of this GPU's 16-bit rate, but enough for a stream, where dp4a kept
//     up to four rows only.  Any order of K serves as long as both operands
//     have the same: a lane's 16 bytes are its K of two MMAs, for the weights and
//     for the rows alike.  The warps' sums meet in shared memory.
// The 7B projection (136 MB of weights): one row 21.5 us (6.3 TB/s, 95 % of the copy
// rate; by the rows kernel 25.0), 8 rows 27.4 us.  Loads of 32 bytes a lane, turns of
// 64 of K and a second turn in flight at fewer blocks per SM made no difference.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "grouped_ring.cuh"
#include "sm103_ptx.cuh"
#include "tc_common.cuh"

namespace swiglu {

struct Int8RowsParams {
  const int8_t *A, *W1, *W2;
  const float *sa, *s1, *s2;
  const int32_t *offsets;  // [E + 1], or null: one matrix for all rows
  const int32_t *rows;     // [P] or null
  __nv_bfloat16 *Y;        // [P, N]
  int32_t T, P, E, N, K;
  int32_t col_blocks;
};

// 16 bytes of weights, not kept in L1.
__device__ __forceinline__ static uint4 load_weights16(const int8_t *p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
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

// acc[16 columns x 8 rows] += columns (32 of K) x rows, all signed bytes.
__device__ __forceinline__ static void mma_s8(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Place `row`'s group, found by the whole block: its expert is the one before the
// first bound above it, its first place the largest bound before that one, its end
// that one (bounds are clamped to [0, P] and made not decreasing).
template <int WARPS>
struct FindGroup {
  static constexpr int PER = (kMaxExperts + 32 * WARPS) / (32 * WARPS);  // bounds of a thread
  int bound[PER], first;
  struct Shared {
    int part[2][WARPS], end;
  };
  // The expert, or -1: no expert's place.
  __device__ __forceinline__ int expert(const Int8RowsParams &p, int row, Shared &sm) {
    int above = -p.E - 1;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int i = threadIdx.x + 32 * WARPS * j;
      bound[j] = i <= p.E ? ptx::load(p.offsets + i) : INT32_MIN;
    }
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (bound[j] > row) above = max(above, -static_cast<int>(threadIdx.x + 32 * WARPS * j));
    above = __reduce_max_sync(0xffffffffu, above);
    if ((threadIdx.x & 31) == 0) sm.part[0][threadIdx.x >> 5] = above;
    __syncthreads();
    first = -sm.part[0][0];
#pragma unroll
    for (int i = 1; i < WARPS; ++i) first = min(first, -sm.part[0][i]);
    return first <= p.E ? first - 1 : -1;
  }
  // After expert(), of an expert's place: its group's first place, and its end.
  __device__ __forceinline__ int start(Shared &sm, int &end) {
    int start = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int i = threadIdx.x + 32 * WARPS * j;
      if (i < first) start = max(start, bound[j]);
      if (i == first) sm.end = bound[j];
    }
    start = __reduce_max_sync(0xffffffffu, start);
    if ((threadIdx.x & 31) == 0) sm.part[1][threadIdx.x >> 5] = start;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < WARPS; ++i) start = max(start, sm.part[1][i]);
    end = sm.end;
    return start;
  }
};

// One place a block.
template <bool FUSED, int NC, int WARPS>
__global__ void __launch_bounds__(32 * WARPS) swiglu_int8_token_kernel(const __grid_constant__ Int8RowsParams p) {
  constexpr int MATS = FUSED ? 2 : 1;
  __shared__ typename FindGroup<WARPS>::Shared sm;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = static_cast<int>(blockIdx.x / p.col_blocks);
  const int col0 = (static_cast<int>(blockIdx.x % p.col_blocks) * WARPS + warp) * NC;
  ptx::grid_launch_dependents();
  ptx::grid_dependency_wait();
  const int src = p.rows ? ptx::load(p.rows + row) : row;
  int e = 0;
  if (p.offsets) {
    FindGroup<WARPS> group;
    e = group.expert(p, row, sm);
    if (e < 0) return;
  }
  if (col0 >= p.N) return;
  const bool named = src >= 0 && src < p.T;
  const int8_t *a = p.A + int64_t(named ? src : 0) * p.K + 16 * lane;
  // a column past N repeats the last
  const int8_t *w[MATS][NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int64_t at = (int64_t(e) * p.N + min(col0 + c, p.N - 1)) * p.K + 16 * lane;
    w[0][c] = p.W1 + at;
    if (FUSED) w[MATS - 1][c] = p.W2 + at;
  }
  // lane c finishes column c; its scales are on their way meanwhile
  const bool mine = lane < NC && col0 + lane < p.N;
  float s = 0.0f, s1 = 0.0f, s2 = 0.0f;
  if (mine && named) {
    s = ptx::load(p.sa + src);
    s1 = ptx::load(p.s1 + int64_t(e) * p.N + col0 + lane);
    if (FUSED) s2 = ptx::load(p.s2 + int64_t(e) * p.N + col0 + lane);
  }
  int acc[MATS][NC] = {};
#pragma unroll(NC == 1 ? 4 : 2)
  for (int k = 0; k + 16 * lane < p.K; k += 512) {
    uint4 v[MATS][NC];
#pragma unroll
    for (int m = 0; m < MATS; ++m)
#pragma unroll
      for (int c = 0; c < NC; ++c) v[m][c] = load_weights16(w[m][c] + k);
    const uint4 x = ptx::load(reinterpret_cast<const uint4 *>(a + k));
#pragma unroll
    for (int m = 0; m < MATS; ++m)
#pragma unroll
      for (int c = 0; c < NC; ++c) acc[m][c] = dot16(v[m][c], x, acc[m][c]);
  }
  __syncwarp();
  // (a lane's sum stays below 2^31 up to the largest K, the warp's for K < 2^17)
  const bool wide = p.K >= 1 << 17;
  float z[MATS] = {};
#pragma unroll
  for (int m = 0; m < MATS; ++m)
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      float sum;
      if (!wide) {
        sum = static_cast<float>(__reduce_add_sync(0xffffffffu, acc[m][c]));
      } else {
        long long t = acc[m][c];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
        sum = static_cast<float>(t);
      }
      z[m] = lane == c ? sum : z[m];
    }
  if (mine) {
    float y = 0.0f;  // a row number that names no row of A gives zeros
    if (named) y = FUSED ? quick_silu_mul(z[0] * s * s1, z[MATS - 1] * s * s2) : z[0] * s * s1;
    p.Y[int64_t(row) * p.N + col0 + lane] = __float2bfloat16_rn(y);
  }
}

// Dense: rows 8 b .. 8 b + 7 for block b.  Grouped, each place has blocks of its
// own, of which those of the first of every eight of an expert do the work.
template <bool FUSED, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, 3) swiglu_int8_rows_kernel(const __grid_constant__ Int8RowsParams p) {
  constexpr int MATS = FUSED ? 2 : 1, ROWS = 8;
  __shared__ typename FindGroup<WARPS>::Shared sm;
  __shared__ int sums[WARPS][MATS][ROWS][16 + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int tile = static_cast<int>(blockIdx.x / p.col_blocks);
  const int col0 = static_cast<int>(blockIdx.x % p.col_blocks) * 16;
  ptx::grid_launch_dependents();
  ptx::grid_dependency_wait();
  const int row0 = p.offsets ? tile : tile * ROWS;
  // the row of A of place row0 + r, or any where that is past the last place
  auto row_of = [&](int r) {
    const int row = min(row0 + r, p.P - 1);
    return p.rows ? ptx::load(p.rows + row) : row;
  };
  const int src = row_of(g);
  int e = 0, end = p.P;
  FindGroup<WARPS> group;
  if (p.offsets) {
    e = group.expert(p, row0, sm);
    if (e < 0) return;
  }
  // The lane's columns g and g + 8: 16 bytes at K = 16 t, 16 t + 64, ...  A column
  // past N repeats the last.
  const int8_t *w[MATS][2];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int64_t at = (int64_t(e) * p.N + min(col0 + g + 8 * c, p.N - 1)) * p.K + 16 * t;
    w[0][c] = p.W1 + at;
    if (FUSED) w[MATS - 1][c] = p.W2 + at;
  }
  struct Turn {
    uint4 v[MATS][2][2];
  };
  const uint4 zero = make_uint4(0, 0, 0, 0);
  auto load = [&](Turn &s, int k) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool in = k + 64 * h + 16 * t < p.K;
#pragma unroll
      for (int m = 0; m < MATS; ++m)
#pragma unroll
        for (int c = 0; c < 2; ++c) s.v[m][c][h] = in ? load_weights16(w[m][c] + k + 64 * h) : zero;
    }
  };
  Turn turn;
  load(turn, 128 * warp);  // on their way while the group's bounds are found
  if (p.offsets) {
    const int start = group.start(sm, end);
    if ((row0 - start) % ROWS != 0) return;  // another block's
  }
  end = min(min(end, p.P), row0 + ROWS);
  // the thread's result, of row r and column col, and its scales, on their way meanwhile
  const int r = threadIdx.x / 16, col = col0 + threadIdx.x % 16;
  const bool mine = r < ROWS && row0 + r < end && col < p.N;
  const int from = mine ? row_of(r) : -1;
  const bool named = from >= 0 && from < p.T;
  float s = 0.0f, s1 = 0.0f, s2 = 0.0f;
  if (named) {
    const int64_t at = int64_t(e) * p.N + col;
    s = ptx::load(p.sa + from);
    s1 = ptx::load(p.s1 + at);
    if (FUSED) s2 = ptx::load(p.s2 + at);
  }
  // the lane's row g; past the end, zeros
  const bool live = row0 + g < end;
  const int8_t *a = p.A + int64_t(min(max(src, 0), p.T - 1)) * p.K + 16 * t;
  int acc[MATS][4] = {};
  auto multiply = [&](const Turn &s, int k) {
    uint4 x[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      x[h] = live && k + 64 * h + 16 * t < p.K ? ptx::load(reinterpret_cast<const uint4 *>(a + k + 64 * h)) : zero;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int m = 0; m < MATS; ++m) {
        const uint4 &c0 = s.v[m][0][h], &c1 = s.v[m][1][h];
        mma_s8(acc[m], c0.x, c1.x, c0.y, c1.y, x[h].x, x[h].y);
        mma_s8(acc[m], c0.z, c1.z, c0.w, c1.w, x[h].z, x[h].w);
      }
  };
  multiply(turn, 128 * warp);
#pragma unroll(FUSED ? 1 : 2)
  for (int k = 128 * (warp + WARPS); k < p.K; k += 128 * WARPS) {
    load(turn, k);
    multiply(turn, k);
  }
  // a lane holds columns g, g + 8 of rows 2t, 2t + 1
#pragma unroll
  for (int m = 0; m < MATS; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[warp][m][2 * t + (i & 1)][g + 8 * (i >> 1)] = acc[m][i];
  __syncthreads();
  if (mine) {
    float y = 0.0f;  // a row number that names no row of A gives zeros
    if (named) {
      // (a warp's sum stays below 2^31 up to the largest K, the block's perhaps not)
      long long z[MATS] = {};
#pragma unroll
      for (int m = 0; m < MATS; ++m)
#pragma unroll
        for (int v = 0; v < WARPS; ++v) z[m] += sums[v][m][r][threadIdx.x % 16];
      y = static_cast<float>(z[0]) * s * s1;
      if (FUSED) y = quick_silu_mul(y, static_cast<float>(z[MATS - 1]) * s * s2);
    }
    p.Y[int64_t(row0 + r) * p.N + col] = __float2bfloat16_rn(y);
  }
}

}  // namespace swiglu
