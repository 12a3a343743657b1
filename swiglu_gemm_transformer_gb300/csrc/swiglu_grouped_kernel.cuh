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
//   * one tcgen05.mma.cta_group::2 of M = 256 x N rows per K slice of 16; each
//     CTA holds 128 of the M rows: FUSED, 64 columns of W1 and the same 64 of
//     W2; linear, 128 columns of W.  A pair makes 128 or 256 output columns
//     for up to NT rows;
//   * FUSED with two MMAs of M = 128 (gate, up) would put both values of an
//     output into one TMEM lane, but reads the rows' tile from shared memory
//     twice (measured 1.31 PFLOP/s where the linear form ran 1.57: 64 experts x
//     1024 rows, K = 2048); so the gate lanes (0-63) and
//     up lanes (64-127) trade half their values through shared memory;
//   * weights are loaded MN-major straight from the row-major [E, K, N]
//     tensors through 3-D tensor maps, whose K extent ends at each expert's
//     last row, so a ragged K step never multiplies the next expert's
//     weights;
//   * each CTA loads its half of the tile's rows with TMA: gathered rows four
//     at a time (gather4), a full dense half in one box, a part of one in boxes
//     of 32 rows.  Several warps issue them, one thread each, chosen with
//     elect.sync: issued by lane 0 of one warp they took about 50 ns apiece
//     (gate/up with rows at 64 experts x 1024 rows, K = 2048, N = 1024: 1118 us;
//     rows copied with cp.async instead 374 us; four warps like this 366 us, eight
//     320 us, sixteen 313 us, dense rows 298 us: bursts of ten calls.  Back to
//     back, under the power cap, eight 371, sixteen 365, dense 346 us);
//   * accumulators are double-buffered in TMEM (NT columns each).
// Unit schedule: every CTA reads `offsets`, counts the row tiles of each
// expert, and the pairs take the units (expert, row tile, column tile) in
// turn; the rows of an expert are split evenly over its row tiles, in steps
// of 32.  Within an expert, GROUP row tiles walk the column tiles together,
// so that they share the weights in L2.  A warp of its own finds the units,
// 32 at a time (one per lane), and hands them to the other roles through a
// ring in shared memory: found by each role for itself, a unit cost about
// 2 us between two main loops.
// SPLIT: for calls of so few units that most SMs would stand idle.  A K step of
// 64 takes a pair about 0.16 us however few rows it has (the MMA's time for 256
// weight rows), so a cluster of several pairs shares one unit: each takes a
// slice of K, and the first pair adds the others' FP32 sums, in order, from its
// shared memory (the ring, idle by then).  At most one unit per cluster.
// Every wait is bounded as in the other kernels.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include "grouped_units.h"
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
  int32_t pairs, kb_per_pair;  // SPLIT: pairs of a cluster, K steps of each
  uint64_t timeout_ns;
  uint32_t *err;
};

// NT: most rows of one tile (MMA N).
template <bool FUSED_, int NT_, bool SPLIT_ = false>
struct GroupedCfg {
  static constexpr bool FUSED = FUSED_;
  static constexpr bool SPLIT = SPLIT_;
  static constexpr int MAX_PAIRS = 4;            // SPLIT: pairs of a cluster
  static constexpr int NT = NT_;
  static constexpr int BK = 64;
  static constexpr int COLS = FUSED ? 64 : 128;  // output columns per CTA
  static constexpr int ATOM_BYTES = 64 * 64 * 2; // one 64-column x 64-K weight box
  static constexpr int W_BYTES = 2 * ATOM_BYTES; // W1 | W2, or two boxes of W
  static constexpr int A_BYTES = NT / 2 * BK * 2;
  static constexpr int STAGE_BYTES = W_BYTES + A_BYTES;
  static constexpr int STAGES = (208 * 1024) / STAGE_BYTES;
  static constexpr int EPI_WARPS = 8;
  // one epilogue warp's block: the 16 x 32 FP32 values its partner gives it
  // (FUSED), then the 16 rows x 32 columns BF16 it stores, rows 80 bytes apart
  // (16-byte reads of eight rows then touch every bank once)
  static constexpr int STG_PITCH = 80;
  static constexpr int STG_BYTES = 16 * 32 * 4;
  static constexpr int STG_OFF = STAGES * STAGE_BYTES;
  static constexpr int TAB_OFF = STG_OFF + EPI_WARPS * STG_BYTES;
  static constexpr int TAB_BYTES = 2 * (kMaxExperts + 1) * 4;
  static constexpr int UNIT_OFF = (TAB_OFF + TAB_BYTES + 15) / 16 * 16;  // two blocks of 32 units
  static constexpr int BAR_OFF = UNIT_OFF + 2 * 32 * 16;
  static constexpr int NUM_BARS = 2 * STAGES + 9;
  static constexpr int SMEM_BYTES = BAR_OFF + NUM_BARS * 8 + 16 + 1024;
  static constexpr int PRODUCER_WARP = EPI_WARPS;
  static constexpr int MMA_WARP = EPI_WARPS + 1;
  static constexpr int ROW_WARP = EPI_WARPS + 2;  // first of the warps that load rows
  // 16 where a stage takes 32 gathers per CTA (8192 tokens, 8 of 64 experts, K =
  // 2048, ragged groups: 335 us, with 8 warps 343, in bursts), 8 where it takes 16
  // (one token's 8 experts 14.3 us, with 16 warps 14.6; weights in L2 10.9 and
  // 11.6; 61 tokens 70.7 and 71.3).  The linear form always has 8: a block's down
  // product has dense rows, and with `rows` it is 8 % slower (8192 tokens, 64
  // experts, K = 1024, N = 2048: 212 us against 197).
  static constexpr int ROW_WARPS = FUSED && NT == 256 ? 16 : 8;
  static constexpr int UNIT_WARP = ROW_WARP + ROW_WARPS;
  static constexpr int THREADS = 32 * (UNIT_WARP + 1);
  static_assert(NT / 8 % ROW_WARPS == 0, "gathers split evenly");
  static constexpr int MMA_M = 256;
  static constexpr int ACC_COLS = NT;  // TMEM columns of one accumulator buffer
  static constexpr int GROUP = 8;
  static_assert(NT == 128 || NT == 256, "rows of a tile");
  static_assert(!SPLIT || (MAX_PAIRS - 1) * NT * 128 * 4 <= STAGES * STAGE_BYTES, "sums fit the ring");
  static_assert(STAGES >= 4, "pipeline depth");
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
};

// Named barrier over `threads` threads that returns whether all of them say so.
__device__ __forceinline__ static bool bar_all(int id, int threads, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred a, b;\n\t"
      "setp.ne.u32 a, %3, 0;\n\t"
      "barrier.cta.red.and.pred b, %1, %2, a;\n\t"
      "selp.u32 %0, 1, 0, b;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(threads), "r"(ok ? 1u : 0u)
      : "memory");
  return r != 0;
}

// The units of one role, in order.  Every lane of the role's warp calls
// next() (or one lane alone, for a role of one lane: ALONE).
template <bool ALONE>
class GroupedUnits {
 public:
  __device__ GroupedUnits(const GroupedUnit *ring, uint32_t full, uint32_t empty,
                          const GroupedParams &p, volatile int *abort_flag)
      : ring_(ring), full_(full), empty_(empty), p_(p), abort_(abort_flag) {}
  // False at the end, or when a wait gave up (ok then false).
  __device__ bool next(GroupedUnit &u, bool &ok) {
    const uint32_t block = i_ >> 5;
    if ((i_ & 31u) == 0u) {
      ok = wait_bar(full_ + 8u * (block & 1u), (block >> 1) & 1u, p_.timeout_ns, abort_, p_.err,
                    WAIT_SCHED_FULL);
      if (!ALONE) ok = __all_sync(0xffffffffu, ok);
      if (!ok) return false;
    }
    const int4 v = *reinterpret_cast<const int4 *>(ring_ + (i_ & 63u));
    u.row0 = v.x, u.end = v.y, u.e = v.z, u.nb = v.w;
    if ((i_ & 31u) == 31u) {  // the block has been read
      if (!ALONE) __syncwarp();
      if (ALONE || (threadIdx.x & 31u) == 0u) ptx::mbar_arrive(empty_ + 8u * (block & 1u));
    }
    ++i_;
    return u.row0 >= 0;
  }

 private:
  const GroupedUnit *ring_;
  uint32_t full_, empty_, i_ = 0;
  const GroupedParams &p_;
  volatile int *abort_;
};

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
    swiglu_grouped_kernel(const __grid_constant__ CUtensorMap tmA,   // dense: boxes of 32 rows; gathered: one row
                          const __grid_constant__ CUtensorMap tmA2,  // dense: boxes of NT / 2 rows
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
  const uint32_t unitf_bar = bars + 8u * (2 * C::STAGES + 5);  // two each
  const uint32_t unite_bar = bars + 8u * (2 * C::STAGES + 7);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::BAR_OFF + C::NUM_BARS * 8);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  int *off = reinterpret_cast<int *>(smem + C::TAB_OFF);  // [E + 1] group bounds
  int *tiles = off + (kMaxExperts + 1);                   // [E + 1] row tiles before expert e

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t crank = ptx::cluster_ctarank();
  const uint32_t lead = C::SPLIT ? crank & ~1u : 0u;  // cluster rank of this pair's leader
  const uint32_t rank = crank - lead;                 // 0 = the pair's leader
  const uint16_t both = static_cast<uint16_t>(0x3u << lead);  // the pair's CTAs, as a mask
  const int kb0 = C::SPLIT ? static_cast<int>(lead >> 1) * p.kb_per_pair : 0;
  const int kb1 = C::SPLIT ? min(p.num_k_blk, kb0 + p.kb_per_pair) : p.num_k_blk;
  const int cid = static_cast<int>(ptx::cluster_id_x());
  const int ncl = static_cast<int>(ptx::num_clusters_x());

  const bool gather = p.rows != nullptr;
  if (warp == C::PRODUCER_WARP && lane == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      ptx::mbar_init(full_bar(s), 1 + 2 * (gather ? C::ROW_WARPS : 1));
      ptx::mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(accf_bar(b), 1);
      ptx::mbar_init(acce_bar(b), 2 * C::EPI_WARPS);
    }
    ptx::mbar_init(drain_bar, 1);
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(unitf_bar + 8u * b, 1);
      // readers of the units: epilogue warps, warps that copy rows, the weights'
      // thread and, in the leader, the MMA's
      ptx::mbar_init(unite_bar + 8u * b,
                     C::EPI_WARPS + (gather ? C::ROW_WARPS : 1) + 1 + (rank == 0 ? 1 : 0));
    }
    *abort_flag = 0;
    ptx::fence_barrier_init();
    ptx::prefetch_tmap(&tmA);
    if (!gather) ptx::prefetch_tmap(&tmA2);
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

  GroupedUnit *ring = reinterpret_cast<GroupedUnit *>(smem + C::UNIT_OFF);
  GroupedUnit mine = {-1, -1, 0, 0};  // epilogue: the tile at hand
  bool have = false;                  // SPLIT: its sums are complete

  // ---- epilogue (warps 0-7, both CTAs) ----
  // Warp q (mod 4) reads TMEM lanes [32q, 32q + 32), the tile's rows in the
  // columns.  Linear: lane i is output column 32q + i; FUSED: warps q = 0, 1
  // hold the gate and q = 2, 3 the up values of output columns 32 (q % 2) + i.
  // Per 32 rows (FUSED) or 16 rows (linear) of the tile; warps 0-3 take the
  // even chunks, warps 4-7 the odd ones.
  const int q = warp & 3, h = (warp >> 2) & 1;
  constexpr int CH = C::FUSED ? 32 : 16;
  const bool gate = q < 2;
  const int wcol = C::FUSED ? 32 * (q & 1) : 32 * q;
  uint8_t *stg = smem + C::STG_OFF + warp * C::STG_BYTES;
  // FUSED: warps q and q ^ 2 trade values; the gate warp finishes a chunk's
  // first 16 rows, the up warp the last 16 (named barrier of their 64 threads)
  float *give = reinterpret_cast<float *>(smem + C::STG_OFF + (warp ^ 2) * C::STG_BYTES);
  const int pair_bar = 1 + 2 * h + (q & 1);
  // Finishes and stores one tile, whose accumulator starts at `tacc`; arrives on
  // `release` (cluster address) once the warp has read it.
  auto finish = [&](const GroupedUnit &un, uint32_t tacc, uint32_t release) {
    const int nchunk = un.n() / CH;
    // the lane's column of 8 in the row segments that the warp stores
    const int scol = un.nb * 2 * C::COLS + static_cast<int>(rank) * C::COLS + wcol + (lane & 3) * 8;
    if (h >= nchunk) {
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive_cluster_relaxed(release);
    }
#pragma unroll 1
    for (int c = h; c < nchunk; c += 2) {
      uint32_t v[CH];
      if constexpr (C::FUSED) ptx::tmem_ld32(tacc + c * CH, v);
      else ptx::tmem_ld16(tacc + c * CH, v);
      ptx::tmem_wait_ld();
      ptx::reg_fence(v);
      if constexpr (C::SPLIT) {
        const float *more = reinterpret_cast<const float *>(smem) + c * CH * 128 + q * 32 + lane;
        for (int s = 1; s < p.pairs; ++s, more += C::NT * 128)
#pragma unroll
          for (int i = 0; i < CH; ++i)
            v[i] = __float_as_uint(__uint_as_float(v[i]) + more[i * 128]);
      }
      if (c + 2 >= nchunk) {
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_cluster_relaxed(release);
      }
      float y[16];
      if constexpr (C::FUSED) {
        if (c != h) asm volatile("bar.sync %0, 64;" ::"r"(pair_bar) : "memory");
#pragma unroll
        for (int i = 0; i < 16; ++i)
          give[i * 32 + lane] = __uint_as_float(gate ? v[16 + i] : v[i]);
        asm volatile("bar.sync %0, 64;" ::"r"(pair_bar) : "memory");
        const float *got = reinterpret_cast<const float *>(stg);
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = got[i * 32 + lane];
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 16; ++i)
          y[i] = gate ? silu_mul(__uint_as_float(v[i]), y[i])
                      : silu_mul(y[i], __uint_as_float(v[16 + i]));
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = __uint_as_float(v[i]);
      }
      __nv_bfloat16 *sp = reinterpret_cast<__nv_bfloat16 *>(stg) + lane;
#pragma unroll
      for (int i = 0; i < 16; ++i) sp[i * (C::STG_PITCH / 2)] = __float2bfloat16_rn(y[i]);
      __syncwarp();
      const int row0 = un.row0 + c * CH + (C::FUSED && !gate ? 16 : 0);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int t = j * 8 + (lane >> 2);
        const int row = row0 + t;
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
  };


  if (warp == C::UNIT_WARP) {
    // ------------------------------------------------------------ unit finder
    // Group bounds and row-tile counts.  The bounds are clamped to [0, P] and
    // made monotone, so that no value of `offsets` reaches past Y.
    int top = 0, sum = 0;
    constexpr int AHEAD = 4;  // loads in flight: each is a trip to memory
    int raw[AHEAD];
    for (int e0 = 0; e0 <= p.E; e0 += 32) {
      const int e = e0 + lane, slot = (e0 / 32) % AHEAD;
      if (slot == 0) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
          raw[i] = e + 32 * i <= p.E ? __ldg(p.offsets + e + 32 * i) : 0;
      }
      int v = raw[0];
#pragma unroll
      for (int i = 1; i < AHEAD; ++i) v = slot == i ? raw[i] : v;
      v = e <= p.E ? min(max(v, 0), p.P) : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int w = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v = max(v, w);
      }
      v = max(v, top);
      const int prev = __shfl_up_sync(0xffffffffu, v, 1);
      // row tiles of expert e - 1
      int t = e >= 1 && e <= p.E ? row_tiles<C::NT>(v - (lane == 0 ? top : prev)) : 0;
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
    __syncwarp();
    for (uint32_t block = 0;; ++block) {
      const bool ok = wait_bar(unite_bar + 8u * (block & 1u), ((block >> 1) & 1u) ^ 1u,
                               block_limit(p.timeout_ns), abort_flag, p.err, WAIT_SCHED_EMPTY);
      if (!__all_sync(0xffffffffu, ok)) break;
      const GroupedUnit r = grouped_unit<C::GROUP>(cid + (int64_t(block) * 32 + lane) * ncl, off,
                                                   tiles, p.E, p.num_n_blk);
      *reinterpret_cast<int4 *>(ring + 32 * (block & 1u) + lane) = make_int4(r.row0, r.end, r.e, r.nb);
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(unitf_bar + 8u * (block & 1u));
      if (__any_sync(0xffffffffu, r.row0 < 0)) break;
    }
  } else if (warp == C::PRODUCER_WARP) {
    // ------------------------------------------------------------ weights (both CTAs)
    if (ptx::elect_one()) {
      uint32_t stage = 0, phase = 0, issued = 0;
      bool ok = true;
      GroupedUnits<true> units(ring, unitf_bar, unite_bar, p, abort_flag);
      GroupedUnit un;
      while (ok && units.next(un, ok)) {
        const int col0 = un.nb * 2 * C::COLS + static_cast<int>(rank) * C::COLS;
        const uint32_t row_bytes = un.row_bytes(0, gather) + un.row_bytes(1, gather);
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!wait_bar(empty_bar(stage), phase ^ 1u, p.timeout_ns, abort_flag, p.err,
                        WAIT_PRODUCER_EMPTY)) {
            ok = false;
            break;
          }
          const uint32_t sw = base + stage * C::STAGE_BYTES;
          const uint32_t fb = ptx::mapa_shared(full_bar(stage), lead);
          // the bytes of both CTAs, weights and rows
          if (rank == 0) ptx::mbar_arrive_expect_tx(full_bar(stage), 2 * C::W_BYTES + row_bytes);
          ptx::tma_load_3d_pair(sw, &tmW1, fb, col0, kb * C::BK, un.e);
          if (C::FUSED)
            ptx::tma_load_3d_pair(sw + C::ATOM_BYTES, &tmW2, fb, col0, kb * C::BK, un.e);
          else
            ptx::tma_load_3d_pair(sw + C::ATOM_BYTES, &tmW1, fb, col0 + 64, kb * C::BK, un.e);
          ++issued;
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
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
  } else if (warp >= C::ROW_WARP) {
    // ------------------------------------------------------------ rows (both CTAs)
    // Dense rows are copied by the first of these warps alone, gathered rows by
    // all of them; the rows of the MMA's N past the tile's end are not copied
    // (their products, of whatever the stage held before, are not stored).  A
    // tile of few rows leaves some threads without a copy, and a thread that
    // only waited for the stages could miss a phase; so each of them also
    // arrives on the stage's "full" barrier.
    const int w = warp - C::ROW_WARP;
    if ((gather || w == 0) && ptx::elect_one()) {
      constexpr int PER = C::NT / 8 / C::ROW_WARPS;  // gathers of a warp per stage
      uint32_t stage = 0, phase = 0;
      bool ok = true;
      GroupedUnits<true> units(ring, unitf_bar, unite_bar, p, abort_flag);
      GroupedUnit un;
      while (ok && units.next(un, ok)) {
        const int row0 = un.row0 + static_cast<int>(rank) * (un.n() >> 1);
        const int rows = un.rows_of(rank);
        // the last group of four repeats the tile's last row
        int idx[PER][4];
        if (gather) {
#pragma unroll
          for (int j = 0; j < PER; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int at = min(row0 + 4 * (w + j * C::ROW_WARPS) + i, un.end - 1);
              idx[j][i] = min(max(__ldg(p.rows + at), 0), p.T - 1);
            }
        }
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!wait_bar(empty_bar(stage), phase ^ 1u, p.timeout_ns, abort_flag, p.err,
                        WAIT_PRODUCER_EMPTY)) {
            ok = false;
            break;
          }
          const uint32_t sa = base + stage * C::STAGE_BYTES + C::W_BYTES;
          const uint32_t fb = ptx::mapa_shared(full_bar(stage), lead);
          ptx::mbar_arrive_cluster_relaxed(fb);
          if (gather) {
#pragma unroll
            for (int j = 0; j < PER; ++j) {
              const int g = w + j * C::ROW_WARPS;
              if (4 * g < rows)
                ptx::tma_gather4_pair(sa + g * 512, &tmA, fb, kb * C::BK, idx[j][0], idx[j][1],
                                      idx[j][2], idx[j][3]);
            }
          } else if (rows > C::NT / 2 - 32) {
            ptx::tma_load_2d_pair(sa, &tmA2, fb, kb * C::BK, row0);
          } else {
            for (int i = 0; i < rows; i += 32)
              ptx::tma_load_2d_pair(sa + i * 128, &tmA, fb, kb * C::BK, row0 + i);
          }
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) spin_ns(100000);  // aborted: copies already in flight into this CTA land
    }
    __syncwarp();
  } else if (warp == C::MMA_WARP) {
    // ------------------------------------------------------------ MMA issuer (leader only)
    if (rank == 0 && ptx::elect_one()) {
      uint32_t stage = 0, phase = 0, abuf = 0, aphase = 0;
      bool ok = true;
      GroupedUnits<true> units(ring, unitf_bar, unite_bar, p, abort_flag);
      GroupedUnit un;
      while (ok && units.next(un, ok)) {
        const uint32_t idesc = ptx::idesc_bf16(C::MMA_M, un.n(), true, false);
        if (!wait_bar(acce_bar(abuf), aphase ^ 1u, p.timeout_ns, abort_flag, p.err,
                      WAIT_MMA_ACC_EMPTY))
          break;
        ptx::tc_fence_after();
        const uint32_t d = tmem_base + abuf * C::ACC_COLS;
        for (int kb = kb0; kb < kb1; ++kb) {
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
            const uint32_t acc = kb != kb0 || kk != 0 ? 1u : 0u;
            const uint64_t wdesc = ptx::smem_desc(sw + kk * 2048, C::ATOM_BYTES, 1024, ptx::SW_128B);
            const uint64_t rdesc = ptx::smem_desc(sa + kk * 32, 16, 1024, ptx::SW_128B);
            ptx::mma_f16_pair(d, wdesc, rdesc, idesc, acc);
          }
          ptx::mma_commit_pair_mc(empty_bar(stage), both);
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        ptx::mma_commit_pair_mc(accf_bar(abuf), both);
        if (++abuf == 2) {
          abuf = 0;
          aphase ^= 1u;
        }
      }
      ptx::mma_commit_pair_mc(drain_bar, static_cast<uint16_t>(0x1u << lead));
      wait_quiet(drain_bar, 0, p.timeout_ns);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    uint32_t abuf = 0, aphase = 0;
    GroupedUnits<false> units(ring, unitf_bar, unite_bar, p, abort_flag);
    // the next unit, its sums complete; false at the end, or when a wait gave up
    auto take = [&] {
      bool ok = true;
      if (!units.next(mine, ok)) return false;
      ok = wait_bar(accf_bar(abuf), aphase, p.timeout_ns, abort_flag, p.err, WAIT_EPI_ACC_FULL);
      return __all_sync(0xffffffffu, ok) != 0;
    };
    if constexpr (C::SPLIT) {  // the only unit: its sums meet after the roles
      have = take();
    } else {
      finish_together(
          take, [&](bool ok) { return C::FUSED ? bar_all(pair_bar, 64, ok) : ok; },
          [&] {
            ptx::tc_fence_after();
            finish(mine, tmem_base + (static_cast<uint32_t>(q * 32) << 16) + abuf * C::ACC_COLS,
                   ptx::mapa_shared(acce_bar(abuf), lead));
            if (++abuf == 2) {
              abuf = 0;
              aphase ^= 1u;
            }
          });
    }
  }

  if constexpr (C::SPLIT) {
    // The pairs' sums: every copy into the first pair's ring and every MMA that
    // reads it has completed, the others' epilogue warps write theirs there,
    // and the first pair finishes the tile.
    ptx::tc_fence_before();
    __syncwarp();
    ptx::cluster_sync();
    ptx::tc_fence_after();
    const uint32_t tacc = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
    if (have && lead != 0) {
      const uint32_t to = ptx::mapa_shared(base, rank) +
                          ((lead / 2 - 1) * C::NT * 128 + q * 32 + lane) * 4;
      const int nchunk = mine.n() / CH;
#pragma unroll 1
      for (int c = h; c < nchunk; c += 2) {
        uint32_t v[CH];
        if constexpr (C::FUSED) ptx::tmem_ld32(tacc + c * CH, v);
        else ptx::tmem_ld16(tacc + c * CH, v);
        ptx::tmem_wait_ld();
        ptx::reg_fence(v);
#pragma unroll
        for (int i = 0; i < CH; ++i) ptx::st_shared_cluster_u32(to + (c * CH + i) * 512, v[i]);
      }
    }
    __syncwarp();
    ptx::cluster_sync();
    if (warp < C::EPI_WARPS && lead == 0) {
      if (C::FUSED) have = bar_all(pair_bar, 64, have);
      if (have) finish(mine, tacc, ptx::mapa_shared(acce_bar(0), lead));
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
