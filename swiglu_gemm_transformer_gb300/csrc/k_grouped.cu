// k_grouped.cu -- launcher and C entry points of the products grouped by
// expert (swiglu_grouped_kernel.cuh).
#include <algorithm>
#include <cstring>

#include "launch.h"
#include "swiglu.h"
#include "swiglu_grouped_kernel.cuh"

namespace swiglu {
namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct GroupedLaunch {
  CUtensorMap a, a2, w1, w2;
  GroupedParams p;
  int64_t units;  // most units the call can have
  int device;
  uint64_t ctx_gen;
  cudaStream_t stream;
};

template <class C>
cudaError_t launch_grouped(GroupedLaunch &gl) {
  static PerDeviceOnce once;
  static int max_clusters[64] = {0};
  auto kern = swiglu_grouped_kernel<C>;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(C::THREADS, 1, 1);
  cfg.dynamicSmemBytes = C::SMEM_BYTES;
  cfg.stream = gl.stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;  // the occupancy query takes the cluster shape only
  if (C::SPLIT) attr[0].val.clusterDim.x = 2 * gl.p.pairs;
  if (once.needed(gl.device, gl.ctx_gen)) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         C::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    if (!C::SPLIT) {
      cfg.gridDim = dim3(2 * 64, 1, 1);
      int n = 0;
      e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
      if (e != cudaSuccess) return e;
      if (n < 1) return cudaErrorInvalidConfiguration;
      max_clusters[gl.device & 63] = n;
    }
    once.done(gl.device, gl.ctx_gen);
  }
  // SPLIT: a cluster per unit; else a persistent grid of pairs
  const int64_t clusters =
      C::SPLIT ? gl.units : std::min<int64_t>(gl.units, max_clusters[gl.device & 63]);
  cfg.gridDim = dim3(unsigned(clusters) * attr[0].val.clusterDim.x, 1, 1);
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, gl.a, gl.a2, gl.w1, gl.w2, gl.p);
}

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;
// Places and columns: the last tile's bounds, up to 256 past them, are 32-bit too.
constexpr int64_t kMaxTiled = kMaxDim - 256;

// W2 == nullptr: the linear form.
int run_grouped(const void *A, const void *W1, const void *W2, bool fused, const int32_t *offsets,
                const int32_t *rows, void *Y, int64_t T, int64_t P, int64_t E, int64_t N,
                int64_t K, void *stream) {
  if (T < 0 || P < 0 || E < 1 || N < 0 || K < 0) return SWIGLU_ERR_INVALID_ARG;
  if (!rows && T != P) return SWIGLU_ERR_INVALID_ARG;
  if (T > kMaxDim || P > kMaxTiled || N > kMaxTiled || K > kMaxDim || E > kMaxExperts)
    return SWIGLU_ERR_UNSUPPORTED;
  if (P == 0 || N == 0) return SWIGLU_OK;
  // one expert's matrix: the tensor map's largest stride is 2^40 bytes
  if (uint64_t(N) * uint64_t(K) >= uint64_t(1) << 39) return SWIGLU_ERR_UNSUPPORTED;
  if (!Y || !offsets) return SWIGLU_ERR_INVALID_ARG;
  if (K > 0 && (!W1 || (fused && !W2) || (T > 0 && !A))) return SWIGLU_ERR_INVALID_ARG;
  if (!ptr_aligned(Y, 16) || !ptr_aligned(offsets, 4) || !ptr_aligned(rows, 4))
    return SWIGLU_ERR_MISALIGNED;
  if (K > 0 && (!ptr_aligned(A, 16) || !ptr_aligned(W1, 16) || !ptr_aligned(W2, 16)))
    return SWIGLU_ERR_MISALIGNED;
  if (N % 8 != 0 || K % 8 != 0) return SWIGLU_ERR_MISALIGNED;
  const uint64_t y_bytes = uint64_t(P) * N * 2, w_bytes = uint64_t(E) * K * N * 2;
  if (ranges_overlap(Y, y_bytes, A, uint64_t(T) * K * 2) ||
      ranges_overlap(Y, y_bytes, W1, w_bytes) || ranges_overlap(Y, y_bytes, W2, w_bytes) ||
      ranges_overlap(Y, y_bytes, offsets, uint64_t(E + 1) * 4) ||
      ranges_overlap(Y, y_bytes, rows, uint64_t(P) * 4))
    return SWIGLU_ERR_INVALID_ARG;

  GroupedLaunch gl;
  std::memset(&gl, 0, sizeof gl);
  GroupedParams &p = gl.p;
  int sms = 0;
  int rc = device_info(&p.err, &sms, &p.timeout_ns, &gl.ctx_gen);
  if (rc != SWIGLU_OK) return rc;
  gl.stream = static_cast<cudaStream_t>(stream);
  // every product is zero: no rows to name, or no K
  if (K == 0 || T == 0)
    return cudaMemsetAsync(Y, 0, y_bytes, gl.stream) == cudaSuccess ? SWIGLU_OK : SWIGLU_ERR_CUDA;
  if (cudaGetDevice(&gl.device) != cudaSuccess) return SWIGLU_ERR_CUDA;

  p.num_k_blk = int32_t(ceil_div(K, 64));
  p.num_n_blk = int32_t(ceil_div(N, fused ? 128 : 256));
  auto units = [&](int rows_per_tile) {
    return (std::min(E, P) + P / rows_per_tile) * p.num_n_blk;
  };
  // Few units and enough K to share: several pairs to a unit.  A cluster of four
  // or eight CTAs fits the GPU 36 or 15 times.  One token, in a graph: down of 2
  // of 8 experts of the 0.5B shape (4864 x 896) 17.0 -> 8.9 us, of the 7B shape
  // (18944 x 3584) 56 -> 43, gate/up of 2 of 64 experts (2048 x 1024) 11.1 -> 9.8;
  // at 17 K steps as fast as without.  With 100 rows an expert the sums to add
  // cost more: 16 K steps 9.0 us without and 11.1 with.
  const int64_t few = units(128);
  const int least = P > 32 * E ? 32 : 16;  // K steps
  const int pairs = few > 36 || p.num_k_blk < least ? 1 : few > 15 ? 2 : 4;
  // Tiles of up to 256 rows read each weight once per 256 rows; tiles of up to
  // 128 rows leave shared memory for two more stages, which is what counts
  // where a group has few rows and the weights' stream is the cost.  Gate/up of
  // 64 experts, K = 2048, N = 1024, by rows per expert: 64 rows 85.7 us in tiles
  // of 128 and 88.1 in tiles of 256, 128 rows 90.9 and 93.4, 192 rows 115 and
  // 99; ragged groups of 127 rows on average 33 and 32 (8 experts, K = 896,
  // N = 4864).
  const int nt = pairs == 1 && P > 96 * E ? 256 : 128;
  const uint64_t adim[2] = {uint64_t(K), uint64_t(T)}, astr[1] = {uint64_t(K) * 2};
  const uint32_t abox[2] = {64, rows ? 1u : 32u}, abox2[2] = {64, uint32_t(nt / 2)};
  const uint64_t wdim[3] = {uint64_t(N), uint64_t(K), uint64_t(E)};
  const uint64_t wstr[2] = {uint64_t(N) * 2, uint64_t(N) * K * 2};
  const uint32_t wbox[3] = {64, 64, 1};
  rc = encode_bf16_map(&gl.a, A, 2, adim, astr, abox);
  if (!rows && rc == SWIGLU_OK) rc = encode_bf16_map(&gl.a2, A, 2, adim, astr, abox2);
  if (rc == SWIGLU_OK) rc = encode_bf16_map(&gl.w1, W1, 3, wdim, wstr, wbox);
  if (rc == SWIGLU_OK) rc = encode_bf16_map(&gl.w2, fused ? W2 : W1, 3, wdim, wstr, wbox);
  if (rc != SWIGLU_OK) return rc;
  p.offsets = offsets;
  p.rows = rows;
  p.Y = static_cast<__nv_bfloat16 *>(Y);
  p.T = int32_t(T);
  p.P = int32_t(P);
  p.E = int32_t(E);
  p.N = int32_t(N);
  gl.units = units(nt);
  p.pairs = pairs;
  p.kb_per_pair = int32_t(ceil_div(p.num_k_blk, pairs));
  cudaError_t e;
  if (pairs > 1)
    e = fused ? launch_grouped<GroupedCfg<true, 128, true>>(gl)
              : launch_grouped<GroupedCfg<false, 128, true>>(gl);
  else if (fused)
    e = nt == 256 ? launch_grouped<GroupedCfg<true, 256>>(gl) : launch_grouped<GroupedCfg<true, 128>>(gl);
  else
    e = nt == 256 ? launch_grouped<GroupedCfg<false, 256>>(gl) : launch_grouped<GroupedCfg<false, 128>>(gl);
  return e == cudaSuccess ? SWIGLU_OK : SWIGLU_ERR_CUDA;
}

}  // namespace
}  // namespace swiglu

extern "C" int swiglu_fused_grouped(const void *A, const void *W1, const void *W2,
                                    const int32_t *offsets, const int32_t *rows, void *Y, int64_t T,
                                    int64_t P, int64_t E, int64_t N, int64_t K, void *stream) {
  return swiglu::run_grouped(A, W1, W2, true, offsets, rows, Y, T, P, E, N, K, stream);
}

extern "C" int swiglu_linear_grouped(const void *X, const void *W, const int32_t *offsets,
                                     const int32_t *rows, void *Z, int64_t T, int64_t P, int64_t E,
                                     int64_t N, int64_t K, void *stream) {
  return swiglu::run_grouped(X, W, nullptr, false, offsets, rows, Z, T, P, E, N, K, stream);
}
