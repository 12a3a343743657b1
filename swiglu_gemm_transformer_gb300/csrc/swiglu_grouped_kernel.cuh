// swiglu_grouped_kernel.cuh -- matrix products grouped by expert, with ragged
// group sizes, on CTA pairs (sm_103a).
//
// The sparse form of the MLP block (page "Riepilogo Tecnico: Sovrapposizione
// delle Attivazioni a Livello di Tile per l'Inferenza Efficiente di LLM",
// section "Definizione del Problema"): the rows p in
// [offsets[e], offsets[e+1]) belong to expert e and
//     FUSED:  Y[p] = SiLU(a W1[e]) (.) (a W2[e]),   a = A[rows[p]] (or A[p])
//     linear: Z[p] = a W[e].
// The sizes of the groups are known on the device only.
//
// Operand order: the weights are the MMA's M side, the rows its N side
// (transposed product).  A group rarely fills whole 128-row tiles; the MMA's
// N comes in steps of 32, so the product of a tile of n rows costs
// ceil(n / 32) * 32 rows instead of 128 or 256, and a group of one row
// costs little more than its weights' stream.
//   * FUSED: per K slice of 16, two tcgen05.mma.cta_group::2 of M = 128 (64
//     columns of W1, then of W2, in each CTA) x N rows: gate and up of one
//     output column land in the same TMEM lane, 128 columns apart, so the
//     activation needs no exchange between threads.  A pair makes 128 output
//     columns for up to NT rows;
//   * linear: one MMA of M = 256 (128 columns of W in each CTA) x N rows; a
//     pair makes 256 output columns;
//   * weights are loaded MN-major straight from the row-major [E, K, N]
//     tensors through 3-D tensor maps, whose K extent ends at each expert's
//     last row, so a ragged K step never multiplies the next expert's
//     weights; each CTA loads its own half of the tile's rows, by TMA gather4
//     where `rows` names them (one lane per four rows), else by 16-row boxes;
//   * accumulators are double-buffered in TMEM (256 columns each).
// Unit schedule: every CTA reads `offsets`, counts the row tiles of each
// expert, and the pairs take the units (expert, row tile, column tile) in
// turn; the rows of an expert are split evenly over its row tiles, in steps
// of 32.  Within an expert, GROUP row tiles walk the column tiles together,
// so that they share the weights in L2.
// Every wait is bounded as in the other kernels.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include "sm103_ptx.cuh"
#include "tc_common.cuh"

namespace swiglu {

constexpr int kMaxExperts = 1024;

struct GroupedParams {
  const int32_t *offsets;  // [E + 1]
  const int32_t *rows;     // [P] or null
  __nv_bfloat16 *Y;        // [P, N]
  int32_t T, P, E, N;      // rows of A, rows of Y, experts, output columns
  int32_t num_k_blk, num_n_blk;
  uint64_t timeout_ns;
  uint32_t *err;
};

// NT: most rows of one tile (MMA N).
template <bool FUSED_, int NT_>
struct GroupedCfg {
  static constexpr bool FUSED = FUSED_;
  static constexpr int NT = NT_;
  static constexpr int BK = 64;
  static constexpr int COLS = FUSED ? 64 : 128;  // output columns per CTA
  static constexpr int ATOM_BYTES = 64 * 64 * 2; // one 64-column x 64-K weight box
  static constexpr int W_BYTES = 2 * ATOM_BYTES; // W1 | W2, or two boxes of W
  static constexpr int A_BYTES = NT / 2 * BK * 2;
  static constexpr int STAGE_BYTES = W_BYTES + A_BYTES;
  static constexpr int STAGES = (208 * 1024) / STAGE_BYTES;
  static constexpr int EPI_WARPS = 8;
  // one warp's staging block: 16 rows x 32 columns BF16, rows 80 bytes apart
  // (16-byte reads of eight rows then touch every bank once)
  static constexpr int STG_PITCH = 80;
  static constexpr int STG_BYTES = 16 * STG_PITCH;
  static constexpr int STG_OFF = STAGES * STAGE_BYTES;
  static constexpr int TAB_OFF = STG_OFF + EPI_WARPS * STG_BYTES;
  static constexpr int TAB_BYTES = 2 * (kMaxExperts + 1) * 4;
  static constexpr int BAR_OFF = (TAB_OFF + TAB_BYTES + 15) / 16 * 16;
  static constexpr int NUM_BARS = 2 * STAGES + 5;
  static constexpr int SMEM_BYTES = BAR_OFF + NUM_BARS * 8 + 16 + 1024;
  static constexpr int PRODUCER_WARP = EPI_WARPS;
  static constexpr int MMA_WARP = EPI_WARPS + 1;
  static constexpr int THREADS = 32 * (EPI_WARPS + 2);
  static constexpr int MMA_M = FUSED ? 128 : 256;
  static constexpr int UP_COL = 128;   // FUSED: TMEM column offset of the up accumulator
  static constexpr int ACC_COLS = 256; // TMEM columns of one accumulator buffer
  static constexpr int GROUP = 8;
  static_assert(NT % 32 == 0 && NT <= 256, "rows of a tile");
  static_assert(STAGES >= 4, "pipeline depth");
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
};

struct GroupedUnit {
  int e, row0, end, n, nb;  // expert, first row, end of the tile's rows, MMA N, column tile
};

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
    swiglu_grouped_kernel(const __grid_constant__ CUtensorMap tmA,
                          const __grid_constant__ CUtensorMap tmW1,
                          const __grid_constant__ CUtensorMap tmW2,  // FUSED only
                          const GroupedParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *smem = smem_raw + (base - raw);

  const uint32_t bars = base + C::BAR_OFF;
  auto full_bar = [&](int s) { return bars + 8u * s; };
  auto empty_bar = [&](int s) { return bars + 8u * (C::STAGES + s); };
  auto accf_bar = [&](int b) { return bars + 8u * (2 * C::STAGES + b); };
  auto acce_bar = [&](int b) { return bars + 8u * (2 * C::STAGES + 2 + b); };
  const uint32_t drain_bar = bars + 8u * (2 * C::STAGES + 4);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::BAR_OFF + C::NUM_BARS * 8);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  int *off = reinterpret_cast<int *>(smem + C::TAB_OFF);  // [E + 1] group bounds
  int *tiles = off + (kMaxExperts + 1);                   // [E + 1] row tiles before expert e

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = ptx::cluster_ctarank();  // 0 = the pair's leader
  const int cid = static_cast<int>(ptx::cluster_id_x());
  const int ncl = static_cast<int>(ptx::num_clusters_x());

  if (warp == C::PRODUCER_WARP && lane == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      ptx::mbar_init(full_bar(s), 1);
      ptx::mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(accf_bar(b), 1);
      ptx::mbar_init(acce_bar(b), 2 * C::EPI_WARPS);
    }
    ptx::mbar_init(drain_bar, 1);
    *abort_flag = 0;
    ptx::fence_barrier_init();
    ptx::prefetch_tmap(&tmA);
    ptx::prefetch_tmap(&tmW1);
    if (C::FUSED) ptx::prefetch_tmap(&tmW2);
  }
  if (warp == C::MMA_WARP) {
    ptx::tmem_alloc_pair(ptx::smem_u32(tmem_slot), 2 * C::ACC_COLS);
    ptx::tmem_relinquish_pair();
  }
  ptx::tc_fence_before();
  ptx::cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  ptx::grid_launch_dependents();
  ptx::grid_dependency_wait();

  // Group bounds and row-tile counts.  The bounds are clamped to [0, P] and
  // made monotone, so that no value of `offsets` reaches past Y.
  if (warp == 0) {
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
      // row tiles of expert e - 1
      int t = e >= 1 && e <= p.E ? (v - (lane == 0 ? top : prev) + C::NT - 1) / C::NT : 0;
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
  __syncthreads();
  const int64_t num_units = int64_t(tiles[p.E]) * p.num_n_blk;

  auto unit_at = [&](int64_t u) {
    GroupedUnit r;
    // the expert whose row tiles hold tile u / num_n_blk
    const int tt = static_cast<int>(u / p.num_n_blk);
    int lo = 0, hi = p.E;  // tiles[lo] <= tt < tiles[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (tiles[mid] <= tt) lo = mid; else hi = mid;
    }
    const int mt = tiles[lo + 1] - tiles[lo];
    const int local = static_cast<int>(u - int64_t(tiles[lo]) * p.num_n_blk);
    const int per_group = C::GROUP * p.num_n_blk;
    const int g = local / per_group;
    const int first = g * C::GROUP;
    const int span = min(C::GROUP, mt - first);
    const int w = local - g * per_group;
    const int cnt = off[lo + 1] - off[lo];
    // even split in steps of 32 rows; no tile is empty: cnt > (mt - 1) * NT
    const int step = ((cnt + mt - 1) / mt + 31) & ~31;
    r.e = lo;
    r.nb = w / span;
    r.row0 = off[lo] + (first + w % span) * step;
    r.end = min(r.row0 + step, off[lo + 1]);
    r.n = (r.end - r.row0 + 31) & ~31;
    return r;
  };

  if (warp == C::PRODUCER_WARP) {
    // ------------------------------------------------------------ TMA producer (both CTAs)
    uint32_t stage = 0, phase = 0, issued = 0;
    bool ok = true;
    for (int64_t u = cid; ok && u < num_units; u += ncl) {
      const GroupedUnit un = unit_at(u);
      const int half = un.n >> 1;  // rows of this CTA
      const int r0 = un.row0 + static_cast<int>(rank) * half;
      int idx[4] = {0, 0, 0, 0};
      if (p.rows != nullptr && 4 * lane < half) {
        // rows past the tile's end repeat its last one; their products are not stored
#pragma unroll
        for (int j = 0; j < 4; ++j)
          idx[j] = min(max(__ldg(p.rows + min(r0 + 4 * lane + j, un.end - 1)), 0), p.T - 1);
      }
      const int col0 = un.nb * 2 * C::COLS + static_cast<int>(rank) * C::COLS;
      for (int kb = 0; kb < p.num_k_blk; ++kb) {
        ok = wait_bar(empty_bar(stage), phase ^ 1u, p.timeout_ns, abort_flag, p.err,
                      WAIT_PRODUCER_EMPTY);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t sw = base + stage * C::STAGE_BYTES;
        const uint32_t sa = sw + C::W_BYTES;
        const uint32_t fb = ptx::mapa_shared(full_bar(stage), 0);
        if (lane == 0) {
          if (rank == 0)
            ptx::mbar_arrive_expect_tx(full_bar(stage), 2 * C::W_BYTES + un.n * C::BK * 2);
          ptx::tma_load_3d_pair(sw, &tmW1, fb, col0, kb * C::BK, un.e);
          if (C::FUSED)
            ptx::tma_load_3d_pair(sw + C::ATOM_BYTES, &tmW2, fb, col0, kb * C::BK, un.e);
          else
            ptx::tma_load_3d_pair(sw + C::ATOM_BYTES, &tmW1, fb, col0 + 64, kb * C::BK, un.e);
        }
        if (p.rows != nullptr) {
          if (4 * lane < half)
            ptx::tma_gather4_pair(sa + lane * 512, &tmA, fb, kb * C::BK, idx[0], idx[1], idx[2],
                                  idx[3]);
        } else if (16 * lane < half) {
          ptx::tma_load_2d_pair(sa + lane * 2048, &tmA, fb, kb * C::BK, r0 + 16 * lane);
        }
        ++issued;
        if (++stage == C::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (lane == 0) {
      if (ok) {
        // Consume the MMA-completion arrivals still due on this CTA's "empty"
        // barriers, so no multicast arrive targets this CTA after it exits.
        const uint32_t n = issued < (uint32_t)C::STAGES ? issued : (uint32_t)C::STAGES;
        for (uint32_t i = issued - n; i < issued; ++i)
          wait_quiet(empty_bar(i % C::STAGES), (i / C::STAGES) & 1u, p.timeout_ns);
      } else {
        spin_ns(100000);  // aborted: copies already in flight into this CTA land
      }
    }
    __syncwarp();
  } else if (warp == C::MMA_WARP) {
    // ------------------------------------------------------------ MMA issuer (leader only)
    if (lane == 0 && rank == 0) {
      uint32_t stage = 0, phase = 0, abuf = 0, aphase = 0;
      bool ok = true;
      for (int64_t u = cid; ok && u < num_units; u += ncl) {
        const GroupedUnit un = unit_at(u);
        const uint32_t idesc = ptx::idesc_bf16(C::MMA_M, un.n, true, false);
        if (!wait_bar(acce_bar(abuf), aphase ^ 1u, p.timeout_ns, abort_flag, p.err,
                      WAIT_MMA_ACC_EMPTY))
          break;
        ptx::tc_fence_after();
        const uint32_t d = tmem_base + abuf * C::ACC_COLS;
        for (int kb = 0; kb < p.num_k_blk; ++kb) {
          if (!wait_bar(full_bar(stage), phase, p.timeout_ns, abort_flag, p.err, WAIT_MMA_FULL)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint32_t sw = base + stage * C::STAGE_BYTES;
          const uint32_t sa = sw + C::W_BYTES;
#pragma unroll
          for (int kk = 0; kk < C::BK / 16; ++kk) {
            // Weights (MMA A): MN-major 64-column boxes ATOM_BYTES apart, 8-row
            // K groups 1024 bytes apart, 16 K rows = 2048 bytes.  Rows (MMA
            // B): K-major, 128-byte swizzle, 32 bytes of K per MMA.
            const uint32_t acc = kb != 0 || kk != 0 ? 1u : 0u;
            const uint64_t wdesc = ptx::smem_desc(sw + kk * 2048, C::ATOM_BYTES, 1024, ptx::SW_128B);
            const uint64_t rdesc = ptx::smem_desc(sa + kk * 32, 16, 1024, ptx::SW_128B);
            ptx::mma_f16_pair(d, wdesc, rdesc, idesc, acc);
            if (C::FUSED) {
              const uint64_t udesc =
                  ptx::smem_desc(sw + C::ATOM_BYTES + kk * 2048, C::ATOM_BYTES, 1024, ptx::SW_128B);
              ptx::mma_f16_pair(d + C::UP_COL, udesc, rdesc, idesc, acc);
            }
          }
          ptx::mma_commit_pair_mc(empty_bar(stage), 0x3);
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        ptx::mma_commit_pair_mc(accf_bar(abuf), 0x3);
        if (++abuf == 2) {
          abuf = 0;
          aphase ^= 1u;
        }
      }
      ptx::mma_commit_pair_mc(drain_bar, 0x1);
      wait_quiet(drain_bar, 0, p.timeout_ns);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue (warps 0-7, both CTAs)
    // Warp q (mod 4) reads TMEM lanes [32q, 32q + 32).  FUSED: output column
    // 32 (q % 2) + lane, rows of the first (q < 2) or second half of the tile
    // in the TMEM columns; linear: output column 32q + lane, all rows.  Warps
    // 0-3 take the even 16-row chunks, warps 4-7 the odd ones.
    const int q = warp & 3, h = warp >> 2;
    const int wcol = C::FUSED ? 32 * (q & 1) : 32 * q;
    uint8_t *stg = smem + C::STG_OFF + warp * C::STG_BYTES;
    uint32_t abuf = 0, aphase = 0;
    for (int64_t u = cid; u < num_units; u += ncl) {
      const GroupedUnit un = unit_at(u);
      bool ok = wait_bar(accf_bar(abuf), aphase, p.timeout_ns, abort_flag, p.err,
                         WAIT_EPI_ACC_FULL);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      ptx::tc_fence_after();
      const uint32_t tacc = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + abuf * C::ACC_COLS;
      const int half = un.n >> 1;
      const int nchunk = (C::FUSED ? half : un.n) / 16;
      const int rbase = un.row0 + (C::FUSED ? (q >> 1) * half : 0);
      // the lane's column of 8 in the row segments that the warp stores
      const int scol = un.nb * 2 * C::COLS + static_cast<int>(rank) * C::COLS + wcol + (lane & 3) * 8;
      const uint32_t release = ptx::mapa_shared(acce_bar(abuf), 0);
      if (h >= nchunk) {
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_cluster_relaxed(release);
      }
#pragma unroll 1
      for (int c = h; c < nchunk; c += 2) {
        uint32_t g[16], v[16];
        ptx::tmem_ld16(tacc + c * 16, g);
        if (C::FUSED) ptx::tmem_ld16(tacc + C::UP_COL + c * 16, v);
        ptx::tmem_wait_ld();
        ptx::reg_fence(g);
        if (C::FUSED) ptx::reg_fence(v);
        if (c + 2 >= nchunk) {
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive_cluster_relaxed(release);
        }
        __nv_bfloat16 *sp = reinterpret_cast<__nv_bfloat16 *>(stg) + lane;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float y = C::FUSED ? silu_mul(__uint_as_float(g[i]), __uint_as_float(v[i]))
                                   : __uint_as_float(g[i]);
          sp[i * (C::STG_PITCH / 2)] = __float2bfloat16_rn(y);
        }
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int t = j * 8 + (lane >> 2);
          const int row = rbase + c * 16 + t;
          if (row < un.end && scol < p.N) {
            uint4 out = *reinterpret_cast<const uint4 *>(stg + t * C::STG_PITCH + (lane & 3) * 16);
            if (p.rows != nullptr) {
              // a row number that names no row of A gives zeros
              const int src = __ldg(p.rows + row);
              if (src < 0 || src >= p.T) out = make_uint4(0, 0, 0, 0);
            }
            *reinterpret_cast<uint4 *>(p.Y + int64_t(row) * p.N + scol) = out;
          }
        }
        __syncwarp();
      }
      if (++abuf == 2) {
        abuf = 0;
        aphase ^= 1u;
      }
    }
  }

  // Both CTAs have passed their last use of the pair's resources before either
  // frees the tensor memory and leaves (relaxed: only the order of execution
  // matters here).
  ptx::tc_fence_before();
  __syncwarp();
  asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
  asm volatile("barrier.cluster.wait;" ::: "memory");
  if (warp == C::MMA_WARP) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem_base, 2 * C::ACC_COLS);
  }
}

}  // namespace swiglu
