// k_int8.cu -- launcher and C entry points of the products in 8-bit integers,
// dense and grouped by expert, and the kernel that widens the rows' codes to
// FP16 before the tensor-core form.
#include <algorithm>
#include <cstring>

#include "launch.h"
#include "swiglu.h"
#include "swiglu_int8_kernel.cuh"
#include "swiglu_int8_rows_kernel.cuh"

namespace swiglu {
namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;
// Places and columns: the last tile's bounds, up to 256 past them, are 32-bit too.
constexpr int64_t kMaxTiled = kMaxDim - 256;
// A warp of the rows kernel adds 128 * 128 * K / 8 at most, in whole turns of 1024 of K.
constexpr int64_t kMaxK = (int64_t(1) << 20) - 1024;

// One expert's matrix: the tensor map's largest stride is 2^40 bytes.
bool matrix_fits(int64_t N, int64_t K) { return uint64_t(N) * uint64_t(K) < uint64_t(1) << 40; }
// Rows of K and of N are copied in pieces of 16 bytes.
bool whole_pieces(int64_t N, int64_t K) { return N % 8 == 0 && K % 16 == 0; }

struct Int8Call {
  const void *A, *W1, *W2;  // W2 == nullptr: the linear form
  const float *sa, *s1, *s2;
  bool fused, grouped;
  const int32_t *offsets, *rows;
  void *Y;
  int64_t T, P, E, N, K;
  void *workspace;
  uint64_t workspace_bytes;
  void *stream;
};

// One row, or places that hardly share experts: a block for each place.
bool one_block_a_place(int64_t P, int64_t E) { return P == 1 || 4 * P <= E; }

// Whether the kernels for a few rows run.  They read a matrix once for 8 rows (from
// L2 after the first time), the tensor-core form once for 192, but that begins with
// a second kernel and ends with a longer tail, about 4 us together.
// Dense, by tiles of 8 rows and bytes of weights (us, rows | tensor cores): 484 MB 8
// rows 81 | 102, 16 rows 150 | 105; 242 MB 8 rows 44 | 54 (K = 8192), 53 | 49 (K =
// 29568); 136 MB 27.8 | 28.7, 49 | 29; 68 MB 17.8 | 22.1, 20.5 | 22.2; 13 MB 16 rows 6.0 |
// 11.2; 4.4 MB 32 rows 5.7 | 11.8; 8.7 MB 32 rows 9.0 | 9.2.
// Grouped, every place has its blocks of 16 columns, of which those of the first of
// eight of an expert work; a block costs 2 to 2.5 ns, a matrix read once more 0.15 us a MB,
// and the tensor-core form reads large matrices slower, by 0.025 us a MB of each expert used
// (fitted to 330 sizes; the form it takes is 0.3 % slower than the better one on average,
// 14 % at most).  Places at random, in a graph: one expert of 4.2 MB (2048 x 1024,
// gate/up) 16 places 6.1 | 8.2, 32 places 10.2 | 8.2; one of 136 MB 2 places 28.6 | 27.9,
// 32 places 188 | 28; 8 of 8.7 MB (896 x 4864) 8 places 17.2 | 15.8, 16 places 27 | 18.7;
// 8 of 68 MB (18944 x 3584) 24 places 71 | 111, 64 places 119 | 113; 64 of 4.2 MB 32
// places 23.6 | 26.4, 96 places 48.8 | 43.3.
constexpr int64_t kFewPlaces = 128;  // as far as this was measured

bool few_rows(int64_t P, int64_t E, int64_t N, int64_t K, bool fused) {
  const int64_t bytes = N * K * (fused ? 2 : 1), tiles = ceil_div(P, 8);
  if (E > 0) {
    const int64_t blocks = ceil_div(N, 16), used = std::min(E, P);
    if (P > kFewPlaces || P * ceil_div(N, 8) > kMaxDim) return false;
    // twice the nanoseconds that the rows' kernel takes longer, but for those 4 us
    const int64_t longer = (4 * (P - used) + 5 * used) * blocks +
                           (std::max(tiles, used) - used) * bytes * 3 / 10000 - used * bytes / 20000;
    return one_block_a_place(P, E) || longer < 9000;
  }
  return tiles == 1 || (tiles <= 16 && bytes <= 200000000 / (9 * tiles - 11));
}

// The tensor-core form reads FP16 rows: A's, or, where there are fewer places
// than rows, the places'.
uint64_t widened_bytes(int64_t T, int64_t P, int64_t K) { return uint64_t(std::min(T, P)) * K * 2; }

// The rows' FP16 values to the workspace; row r is A's row rows[r] (any row where
// that names none), or r.  Eight codes a lane, so that loads and stores cover whole
// lines, four times over, which keeps enough of them in flight.  Bound by the
// copy rate: 65536 rows of 1024 codes 26.7 us (16 codes a lane in a loop: 36).
constexpr int kWidenTurns = 4;

__global__ void __launch_bounds__(256) widen_rows_kernel(const int8_t *A, const int32_t *rows, __half *out,
                                                         int64_t count, int32_t per_row, int32_t T, bool early) {
  // In this order the product's kernel starts when nothing before this one runs;
  // early: at once, and waits for this one's end itself.
  if (early) ptx::grid_launch_dependents();
  ptx::grid_dependency_wait();
  if (!early) ptx::grid_launch_dependents();
  const int64_t first = int64_t(blockIdx.x) * (256 * kWidenTurns) + threadIdx.x;
  uint2 v[kWidenTurns];
#pragma unroll
  for (int j = 0; j < kWidenTurns; ++j) {
    const int64_t i = first + 256 * j;
    if (i >= count) break;
    int64_t from = i;
    if (rows) {
      const int64_t r = i / per_row;
      from = int64_t(min(max(ptx::load(rows + r), 0), T - 1)) * per_row + (i - r * per_row);
    }
    v[j] = ptx::load(reinterpret_cast<const uint2 *>(A) + from);
  }
#pragma unroll
  for (int j = 0; j < kWidenTurns; ++j) {
    const int64_t i = first + 256 * j;
    if (i >= count) break;
    uint4 o;
    widen4(v[j].x, o.x, o.y);
    widen4(v[j].y, o.z, o.w);
    reinterpret_cast<uint4 *>(out)[i] = o;
  }
}

cudaError_t launch_widen(const Int8Call &c, const int32_t *rows, int64_t n, bool early) {
  const int64_t per_row = c.K / 8, count = n * per_row, blocks = ceil_div(count, 256 * kWidenTurns);
  if (blocks > kMaxDim) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(256);
  cfg.stream = static_cast<cudaStream_t>(c.stream);
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, widen_rows_kernel, static_cast<const int8_t *>(c.A), rows,
                            static_cast<__half *>(c.workspace), count, int32_t(per_row), int32_t(c.T), early);
}

// The kernel `kern` for `tiles` of rows and blocks of `cols` columns.
cudaError_t launch_rows(void (*kern)(Int8RowsParams), Int8RowsParams &p, int64_t tiles, int cols, cudaStream_t s) {
  p.col_blocks = int32_t(ceil_div(p.N, cols));
  if (tiles * p.col_blocks > kMaxDim) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * p.col_blocks));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

// The kernels for a few rows.
cudaError_t run_rows(Int8RowsParams &p, bool fused, int sms, cudaStream_t s) {
  // One row, or places that hardly share experts: a block for each place, whose
  // warps take one, two or four columns of each matrix, as many as leave four blocks
  // to each SM (one row of 18944 x 3584 with four columns 25.1 us, so
  // 15.2; of 4096 x 8192 11.0 and 8.4).  Grouped, two blocks: a block begins with
  // the search for its expert (one token, 8 of 64 experts, 2048 x 1024, gate/up 9.3
  // and 8.5 us, down 7.2 and 5.8).
  if (one_block_a_place(p.P, p.offsets ? p.E : 0)) {
    const int64_t cols = int64_t(p.N) * p.P / (8 * sms * (p.offsets ? 2 : 4));  // of a warp
    if (fused)
      return cols >= 2 ? launch_rows(swiglu_int8_token_kernel<true, 2, 8>, p, p.P, 16, s)
                       : launch_rows(swiglu_int8_token_kernel<true, 1, 8>, p, p.P, 8, s);
    return cols >= 4   ? launch_rows(swiglu_int8_token_kernel<false, 4, 8>, p, p.P, 32, s)
           : cols >= 2 ? launch_rows(swiglu_int8_token_kernel<false, 2, 8>, p, p.P, 16, s)
                       : launch_rows(swiglu_int8_token_kernel<false, 1, 8>, p, p.P, 8, s);
  }
  return launch_rows(fused ? swiglu_int8_rows_kernel<true, 8> : swiglu_int8_rows_kernel<false, 8>, p,
                     p.offsets ? p.P : ceil_div(p.P, 8), 16, s);
}

struct TensorLaunch {
  CUtensorMap a, a2, w1, w2;
  Int8Params p;
  int64_t units;  // most units the call can have
  int device;
  uint64_t ctx_gen;
  cudaStream_t stream;
};

template <class C>
cudaError_t launch_tensor(TensorLaunch &t) {
  static PerDeviceOnce once;
  static int max_clusters[64] = {0};
  auto kern = swiglu_int8_kernel<C>;
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
  cfg.stream = t.stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;  // the occupancy query takes the cluster shape only
  if (C::SPLIT) attr[0].val.clusterDim.x = 2 * t.p.pairs;
  if (once.needed(t.device, t.ctx_gen)) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    if (!C::SPLIT) {
      cfg.gridDim = dim3(2 * 64, 1, 1);
      int n = 0;
      e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
      if (e != cudaSuccess) return e;
      if (n < 1) return cudaErrorInvalidConfiguration;
      max_clusters[t.device & 63] = n;
    }
    once.done(t.device, t.ctx_gen);
  }
  // SPLIT: a cluster per unit; else a persistent grid of pairs
  const int64_t clusters = C::SPLIT ? t.units : std::min<int64_t>(t.units, max_clusters[t.device & 63]);
  cfg.gridDim = dim3(unsigned(clusters) * attr[0].val.clusterDim.x, 1, 1);
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, t.a, t.a2, t.w1, t.w2, t.p);
}

// The tensor-core form.
int run_tensor(const Int8Call &c, uint32_t *err, uint64_t timeout_ns, uint64_t ctx_gen) {
  using Fused = Int8Cfg<true, 192>;
  using Split = Int8Cfg<true, 128, true>;
  TensorLaunch t;
  std::memset(&t, 0, sizeof t);
  t.stream = static_cast<cudaStream_t>(c.stream);
  t.ctx_gen = ctx_gen;
  if (cudaGetDevice(&t.device) != cudaSuccess) return SWIGLU_ERR_CUDA;
  // Rows in the places' order where they are no more than A's; else A's rows, which
  // the kernel gathers.
  const bool gather = c.rows && c.P > c.T;
  const uint64_t R = uint64_t(std::min(c.T, c.P)), E = c.E, N = c.N, K = c.K;
  const int32_t k_blk = int32_t(ceil_div(c.K, Fused::BK)), n_blk = int32_t(ceil_div(c.N, c.fused ? 128 : 256));
  auto units = [&](int nt) { return (c.offsets ? std::min(c.E, c.P) + c.P / nt : ceil_div(c.P, nt)) * n_blk; };
  // Few units and enough K to share: several pairs to a unit.  A cluster of four
  // or eight CTAs fits the GB300 36 or 15 times.  125 rows of 4864 x 896 22.7 -> 13.5
  // us, 128 rows of 3584 x 3584 19.2 -> 13.8, of 2048 x 2048 13.9 -> 11.5; at 8 K
  // steps (64 rows of 1024 x 2048) 9.6 and 9.7.
  const int64_t few = units(Split::NT);
  const int pairs = few > 36 || k_blk < 8 ? 1 : few > 15 ? 2 : Split::MAX_PAIRS;
  // Tiles of up to 128 rows leave shared memory for two more stages of codes, which
  // counts where the weights' stream is the cost.  64 experts, gate/up of 2048 x 1024
  // and down of 1024 x 2048, tiles of 128 | 192: 16 rows an expert 51.4 | 52.2 and
  // 30.0 | 32.1 us, 96 rows 60.8 | 61.7 and 39.0 | 40.3, 128 rows (ragged) 86 | 66 and
  // 47.5 | 42.4; the 7B projection of 128 rows 31.9 | 34.5.
  const int nt = pairs > 1 || c.P <= (c.offsets ? 96 * c.E : Split::NT) ? Split::NT : Fused::NT;
  const uint64_t adim[2] = {K, R}, astr[1] = {K * 2};
  const uint32_t abox[2] = {64, gather ? 1u : 32u}, abox2[2] = {64, uint32_t(nt / 2)};
  const uint64_t wdim[3] = {K, N, E}, wstr[2] = {K, N * K};
  const uint32_t wbox[3] = {Fused::BK, 64, 1};
  int rc = encode_bf16_map(&t.a, c.workspace, 2, adim, astr, abox);  // (16-bit elements)
  if (!gather && rc == SWIGLU_OK) rc = encode_bf16_map(&t.a2, c.workspace, 2, adim, astr, abox2);
  if (rc == SWIGLU_OK) rc = encode_u8_map(&t.w1, c.W1, 3, wdim, wstr, wbox);
  if (rc == SWIGLU_OK) rc = encode_u8_map(&t.w2, c.fused ? c.W2 : c.W1, 3, wdim, wstr, wbox);
  if (rc != SWIGLU_OK) return rc;
  if (launch_widen(c, gather ? nullptr : c.rows, int64_t(R), pairs > 1) != cudaSuccess)
    return SWIGLU_ERR_CUDA;
  Int8Params &p = t.p;
  p.sa = c.sa;
  p.s1 = c.s1;
  p.s2 = c.s2;
  p.offsets = c.offsets;
  p.rows = c.rows;
  p.Y = static_cast<__nv_bfloat16 *>(c.Y);
  p.T = int32_t(c.T);
  p.P = int32_t(c.P);
  p.E = int32_t(c.E);
  p.N = int32_t(c.N);
  p.gather = gather;
  p.num_k_blk = k_blk;
  p.num_n_blk = n_blk;
  p.timeout_ns = timeout_ns;
  p.err = err;
  p.pairs = pairs;
  t.units = units(nt);
  cudaError_t e;
  if (pairs > 1)
    e = c.fused ? launch_tensor<Int8Cfg<true, 128, true>>(t) : launch_tensor<Int8Cfg<false, 128, true>>(t);
  else if (nt == 128)
    e = c.fused ? launch_tensor<Int8Cfg<true, 128>>(t) : launch_tensor<Int8Cfg<false, 128>>(t);
  else
    e = c.fused ? launch_tensor<Int8Cfg<true, 192>>(t) : launch_tensor<Int8Cfg<false, 192>>(t);
  return e == cudaSuccess ? SWIGLU_OK : SWIGLU_ERR_CUDA;
}

int run_int8(const Int8Call &c) {
  const int64_t T = c.T, P = c.P, E = c.E, N = c.N, K = c.K;
  if (T < 0 || P < 0 || E < 1 || N < 0 || K < 0) return SWIGLU_ERR_INVALID_ARG;
  if (!c.rows && T != P) return SWIGLU_ERR_INVALID_ARG;
  if (T > kMaxDim || P > kMaxTiled || N > kMaxTiled || K > kMaxK || E > kMaxExperts)
    return SWIGLU_ERR_UNSUPPORTED;
  if (P == 0 || N == 0) return SWIGLU_OK;
  if (!matrix_fits(N, K)) return SWIGLU_ERR_UNSUPPORTED;
  if (!c.Y || (c.grouped && !c.offsets)) return SWIGLU_ERR_INVALID_ARG;
  if (K > 0 && (!c.W1 || !c.s1 || (c.fused && (!c.W2 || !c.s2)) || (T > 0 && (!c.A || !c.sa))))
    return SWIGLU_ERR_INVALID_ARG;
  if (!ptr_aligned(c.Y, 16) || !ptr_aligned(c.offsets, 4) || !ptr_aligned(c.rows, 4))
    return SWIGLU_ERR_MISALIGNED;
  if (K > 0 && (!ptr_aligned(c.A, 16) || !ptr_aligned(c.W1, 16) || !ptr_aligned(c.W2, 16) ||
                !ptr_aligned(c.sa, 4) || !ptr_aligned(c.s1, 4) || !ptr_aligned(c.s2, 4)))
    return SWIGLU_ERR_MISALIGNED;
  if (!whole_pieces(N, K)) return SWIGLU_ERR_MISALIGNED;
  const uint64_t y_bytes = uint64_t(P) * N * 2, w_bytes = uint64_t(E) * N * K, s_bytes = uint64_t(E) * N * 4;
  if (ranges_overlap(c.Y, y_bytes, c.A, uint64_t(T) * K) || ranges_overlap(c.Y, y_bytes, c.W1, w_bytes) ||
      ranges_overlap(c.Y, y_bytes, c.W2, w_bytes) || ranges_overlap(c.Y, y_bytes, c.sa, uint64_t(T) * 4) ||
      ranges_overlap(c.Y, y_bytes, c.s1, s_bytes) || ranges_overlap(c.Y, y_bytes, c.s2, s_bytes) ||
      ranges_overlap(c.Y, y_bytes, c.offsets, uint64_t(E + 1) * 4) ||
      ranges_overlap(c.Y, y_bytes, c.rows, uint64_t(P) * 4))
    return SWIGLU_ERR_INVALID_ARG;
  const uint64_t need = swiglu_int8_workspace_size(T, P, c.grouped ? E : 0, N, K, c.fused);
  if (need > 0) {
    if (!c.workspace || c.workspace_bytes < need) return SWIGLU_ERR_INVALID_ARG;
    if (!ptr_aligned(c.workspace, 16)) return SWIGLU_ERR_MISALIGNED;
    // (A, W1, W2, scales, offsets, rows and Y; all are read or written after it)
    const void *ptr[9] = {c.A, c.W1, c.W2, c.sa, c.s1, c.s2, c.offsets, c.rows, c.Y};
    const uint64_t len[9] = {uint64_t(T) * K, w_bytes, w_bytes, uint64_t(T) * 4, s_bytes, s_bytes,
                             uint64_t(E + 1) * 4, uint64_t(P) * 4, y_bytes};
    for (int i = 0; i < 9; ++i)
      if (ranges_overlap(c.workspace, need, ptr[i], len[i])) return SWIGLU_ERR_INVALID_ARG;
  }
  uint32_t *err = nullptr;
  int sms = 0;
  uint64_t timeout_ns = 0, gen = 0;
  const int rc = device_info(&err, &sms, &timeout_ns, &gen);
  if (rc != SWIGLU_OK) return rc;
  const cudaStream_t s = static_cast<cudaStream_t>(c.stream);
  // every product is zero: no rows to name, or no K
  if (K == 0 || T == 0)
    return cudaMemsetAsync(c.Y, 0, y_bytes, s) == cudaSuccess ? SWIGLU_OK : SWIGLU_ERR_CUDA;
  Int8RowsParams p = {};
  p.A = static_cast<const int8_t *>(c.A);
  p.W1 = static_cast<const int8_t *>(c.W1);
  p.W2 = static_cast<const int8_t *>(c.W2);
  p.sa = c.sa;
  p.s1 = c.s1;
  p.s2 = c.s2;
  p.offsets = c.offsets;
  p.rows = c.rows;
  p.Y = static_cast<__nv_bfloat16 *>(c.Y);
  p.T = int32_t(T);
  p.P = int32_t(P);
  p.E = int32_t(E);
  p.N = int32_t(N);
  p.K = int32_t(K);
  if (need > 0) return run_tensor(c, err, timeout_ns, gen);
  const cudaError_t e = run_rows(p, c.fused, sms, s);
  return e == cudaSuccess ? SWIGLU_OK : SWIGLU_ERR_CUDA;
}

}  // namespace
}  // namespace swiglu

extern "C" uint64_t swiglu_int8_workspace_size(int64_t T, int64_t P, int64_t E, int64_t N, int64_t K,
                                               int32_t fused) {
  using namespace swiglu;
  if (T < 1 || T > kMaxDim || P < 1 || P > kMaxTiled || E < 0 || E > kMaxExperts || N < 1 || N > kMaxTiled || K < 1 ||
      K > kMaxK || !matrix_fits(N, K) || !whole_pieces(N, K) || (E == 0 && T != P) || few_rows(P, E, N, K, fused != 0))
    return 0;
  return widened_bytes(T, P, K);
}

extern "C" int swiglu_fused_int8(const void *A, const float *a_scale, const void *W1, const float *s1,
                                 const void *W2, const float *s2, void *Y, int64_t M, int64_t N,
                                 int64_t K, void *workspace, uint64_t workspace_bytes, void *stream) {
  return swiglu::run_int8({A, W1, W2, a_scale, s1, s2, true, false, nullptr, nullptr, Y, M, M, 1, N, K,
                           workspace, workspace_bytes, stream});
}

extern "C" int swiglu_linear_int8(const void *X, const float *x_scale, const void *W, const float *w_scale,
                                  void *Z, int64_t M, int64_t N, int64_t K, void *workspace,
                                  uint64_t workspace_bytes, void *stream) {
  return swiglu::run_int8({X, W, nullptr, x_scale, w_scale, nullptr, false, false, nullptr, nullptr, Z, M, M, 1, N, K,
                           workspace, workspace_bytes, stream});
}

extern "C" int swiglu_fused_grouped_int8(const void *A, const float *a_scale, const void *W1,
                                         const float *s1, const void *W2, const float *s2,
                                         const int32_t *offsets, const int32_t *rows, void *Y, int64_t T,
                                         int64_t P, int64_t E, int64_t N, int64_t K, void *workspace,
                                         uint64_t workspace_bytes, void *stream) {
  return swiglu::run_int8({A, W1, W2, a_scale, s1, s2, true, true, offsets, rows, Y, T, P, E, N, K,
                           workspace, workspace_bytes, stream});
}

extern "C" int swiglu_linear_grouped_int8(const void *X, const float *x_scale, const void *W,
                                          const float *w_scale, const int32_t *offsets,
                                          const int32_t *rows, void *Z, int64_t T, int64_t P, int64_t E,
                                          int64_t N, int64_t K, void *workspace, uint64_t workspace_bytes,
                                          void *stream) {
  return swiglu::run_int8({X, W, nullptr, x_scale, w_scale, nullptr, false, true, offsets, rows, Z, T, P, E, N, K,
                           workspace, workspace_bytes, stream});
}
