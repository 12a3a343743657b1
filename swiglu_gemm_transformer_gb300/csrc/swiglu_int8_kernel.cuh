// swiglu_int8_kernel.cuh -- products in 8-bit integers on CTA pairs (sm_103a),
// dense or grouped by expert.
//
//     z[p,n] = sa[p] sw[e,n] sum_k A[p,k] W[e,n,k]         (linear)
//     y[p,n] = SiLU(z1[p,n]) z2[p,n]                       (FUSED)
//
// This GPU multiplies 8-bit integers at a tenth of its 16-bit rate, so the
// codes are widened to FP16 (exact: 11 significant bits) on their way to the
// MMA, whose FP32 sums of their products are exact below 2^24 (beyond, with codes of
// one sign results were off by 1.3 % at K = 2^20 - 1024, by no more than BF16's rounding
// up to 2^17).  As in the
// BF16 grouped kernel the weights are the MMA's M side (256 per pair) and the
// rows its N side, in steps of 32; the units and their finder are the same.
//   * the weights are copied as codes, 128 of K a stage (TMA), half the bytes of
//     16-bit operands, and widened straight into tensor memory, as the MMA's A
//     operand: K-major codes give a thread its lane's K in 16-byte loads, and
//     shared memory, which feeds copies, loads and the MMA's B operand alike, is
//     spared their 16-bit form.  Two groups of four warps take a half of 64 of K
//     each;
//   * the rows come as FP16, widened once per call by a small kernel before this
//     one (k_int8.cu): widened here they cost as many instructions as the
//     weights, once for each column tile (7B projection, 2047 rows: 378 us so, 321
//     with that kernel, before the next point);
//   * accumulators of 192 columns, double-buffered, leave 128 columns for two
//     steps of weights, of 128 of K each.  A buffer of them is freed, filled,
//     announced and read in turn, so the codes are widened before the wait for
//     it.  Steps of 64 (four buffers) were bound by the MMA's thread, which a
//     commit holds up for about 230 cycles: 480 a step however few rows it had (the
//     7B projection 321 us, with steps of 128 306);
//   * FUSED: gate and up of a column lie in lanes 2j and 2j ^ 9 of one warp (odd
//     lanes take the up columns, in an order that keeps the loads of eight
//     lanes on different banks), so shuffles bring them together.
// SPLIT: for calls of so few units that most SMs would stand idle: the pairs of a
// cluster share one unit's K; then each finishes a part of its rows, to whose
// sums it adds the others', in order, from its shared memory (the rings, idle by
// then).  With one pair finishing all 125 rows a call took 15.4 us, 12.8 so.
// Every wait is bounded as in the other kernels, the one for a unit's sums by its K.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "grouped_ring.cuh"
#include "sm103_ptx.cuh"
#include "tc_common.cuh"

namespace swiglu {

struct Int8Params {
  const float *sa, *s1, *s2;  // scales of the rows of A, of W1's and W2's columns [E, N]
  const int32_t *offsets;     // [E + 1], or null: one matrix for all rows
  const int32_t *rows;        // [P] or null
  __nv_bfloat16 *Y;           // [P, N]
  int32_t T, P, E, N;         // rows of A, rows of Y, experts, output columns
  int32_t gather;             // 1: the FP16 rows are A's; 0: they are in the places' order
  int32_t num_k_blk, num_n_blk;  // K steps, column tiles
  int32_t pairs;                 // SPLIT: pairs of a cluster, at most num_k_blk
  uint64_t timeout_ns;
  uint32_t *err;
};

template <bool FUSED_, int NT_, bool SPLIT_ = false>
struct Int8Cfg {
  static constexpr bool FUSED = FUSED_;
  static constexpr bool SPLIT = SPLIT_;
  static constexpr int MAX_PAIRS = 4;            // SPLIT: pairs of a cluster
  static constexpr int NT = NT_;                 // most rows of a tile
  static constexpr int BK = 128;                 // K of a step
  static constexpr int COLS = FUSED ? 64 : 128;  // output columns per CTA
  static constexpr int BOX_BYTES = 64 * BK;      // 64 columns' codes
  static constexpr int W_BYTES = 2 * BOX_BYTES;  // W1 | W2, or two boxes of W
  static constexpr int W_STAGES = NT == 128 ? 8 : 6;
  static constexpr int HALF_BYTES = NT / 2 * 64 * 2;  // the rows' FP16 values, 64 of K
  static constexpr int A_BYTES = 2 * HALF_BYTES;
  static constexpr int A_STAGES = 4;
  static constexpr int BUFS = 2;                 // widened weights, a step each
  static constexpr int EPI_WARPS = 8;
  // one epilogue warp's block: 16 rows x 32 columns BF16 (rows 80 bytes apart:
  // 16-byte reads of eight rows touch every bank once), FUSED 16 x 16 (48 apart)
  static constexpr int STG_PITCH = FUSED ? 48 : 80;
  static constexpr int STG_BYTES = 1280;
  static constexpr int SCALE_BYTES = 96 * 4;     // and the scales of the rows it finishes
  static constexpr int A_OFF = W_STAGES * W_BYTES;
  static constexpr int STG_OFF = A_OFF + A_STAGES * A_BYTES;
  static constexpr int SCALE_OFF = STG_OFF + EPI_WARPS * STG_BYTES;
  static constexpr int TAB_OFF = SCALE_OFF + EPI_WARPS * SCALE_BYTES;
  static constexpr int TAB_BYTES = 2 * (kMaxExperts + 1) * 4;
  static constexpr int UNIT_OFF = (TAB_OFF + TAB_BYTES + 15) / 16 * 16;  // two blocks of 32 units
  static constexpr int BAR_OFF = UNIT_OFF + 2 * 32 * 16;
  static constexpr int NUM_BARS = 2 * W_STAGES + 2 * A_STAGES + BUFS + 9;
  static constexpr int SMEM_BYTES = BAR_OFF + NUM_BARS * 8 + 16 + 1024;
  static constexpr int W_WARP = EPI_WARPS;       // first of those that widen weights
  // Two groups of four: gate/up of 8192 tokens 363 us, three 368, four (and four
  // warps that copy rows) 437; the 7B projection 300 all.
  static constexpr int PRODUCER_WARP = W_WARP + 8;
  static constexpr int MMA_WARP = PRODUCER_WARP + 1;
  static constexpr int UNIT_WARP = MMA_WARP + 1;
  static constexpr int LOAD_WARP = UNIT_WARP + 1;  // first of those that copy rows
  static constexpr int LOAD_WARPS = 8;
  static constexpr int THREADS = 32 * (LOAD_WARP + LOAD_WARPS);
  static constexpr int ACC_COLS = 192;           // TMEM columns of one accumulator buffer
  static constexpr int OP_COL = 2 * ACC_COLS;    // then the widened weights, 64 columns a step
  static constexpr int GROUP = 8;
  static_assert(NT <= ACC_COLS && OP_COL + BUFS * 64 == 512, "tensor memory");
  // (two pairs: one half of the rows from one other; four: a quarter from three)
  static_assert(!SPLIT || NT * 128 * 4 <= STG_OFF, "sums fit the rings");
  static_assert(A_STAGES % BUFS == 0, "one arrival frees rows and weights");
  static_assert(NT / 8 % LOAD_WARPS == 0, "gathers split evenly");
  static_assert(THREADS <= 1024, "threads");
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
};

// Four codes to FP16: with the sign bit flipped (u = q + 128) and 0x64 above it
// a byte is the FP16 number 1024 + u; minus 1152 is q.
__device__ __forceinline__ static void widen4(uint32_t codes, uint32_t &lo, uint32_t &hi) {
  const uint32_t u = codes ^ 0x80808080u;
  const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
  const uint32_t k = 0x64806480u;
  const __half2 x = __hsub2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&k));
  const __half2 y = __hsub2(*reinterpret_cast<const __half2 *>(&b), *reinterpret_cast<const __half2 *>(&k));
  lo = *reinterpret_cast<const uint32_t *>(&x);
  hi = *reinterpret_cast<const uint32_t *>(&y);
}

__device__ __forceinline__ static uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
    swiglu_int8_kernel(const __grid_constant__ CUtensorMap tmA,   // dense: boxes of 32 rows; gathered: one row
                       const __grid_constant__ CUtensorMap tmA2,  // dense: boxes of NT / 2 rows
                       const __grid_constant__ CUtensorMap tmW1,
                       const __grid_constant__ CUtensorMap tmW2,  // linear: W1 again
                       const __grid_constant__ Int8Params p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *smem = smem_raw + (base - raw);

  const uint32_t bars = base + C::BAR_OFF;
  auto full_bar = [&](int s) { return bars + 8u * s; };                    // a stage's codes are there
  auto empty_bar = [&](int s) { return bars + 8u * (C::W_STAGES + s); };   // and have been read
  const uint32_t abars = bars + 8u * 2 * C::W_STAGES;
  auto rows_bar = [&](int s) { return abars + 8u * s; };                   // leader: both CTAs' rows of a step are there
  auto done_bar = [&](int s) { return abars + 8u * (C::A_STAGES + s); };   // the MMA has read the step's operands
  auto op_bar = [&](int b) { return abars + 8u * (2 * C::A_STAGES + b); };  // leader: both CTAs' widened weights
  const uint32_t accf = abars + 8u * (2 * C::A_STAGES + C::BUFS), acce = accf + 16u;  // two each
  const uint32_t unitf_bar = accf + 32u, unite_bar = accf + 48u;                      // two each
  const uint32_t drain_bar = accf + 64u;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::BAR_OFF + C::NUM_BARS * 8);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  int *off = reinterpret_cast<int *>(smem + C::TAB_OFF);  // [E + 1] group bounds
  int *tiles = off + (kMaxExperts + 1);                   // [E + 1] row tiles before expert e
  GroupedUnit *ring = reinterpret_cast<GroupedUnit *>(smem + C::UNIT_OFF);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t crank = ptx::cluster_ctarank();
  const uint32_t lead = C::SPLIT ? crank & ~1u : 0u;  // cluster rank of this pair's leader
  const uint32_t rank = crank - lead;                 // 0 = the pair's leader
  const uint16_t both = static_cast<uint16_t>(0x3u << lead);  // the pair's CTAs, as a mask
  const int kb0 = C::SPLIT ? p.num_k_blk * static_cast<int>(lead >> 1) / p.pairs : 0;
  const int kb1 = C::SPLIT ? p.num_k_blk * static_cast<int>((lead >> 1) + 1) / p.pairs : p.num_k_blk;
  const bool gather = p.gather != 0;
  const int loaders = gather ? C::LOAD_WARPS : 1;

  if (warp == C::PRODUCER_WARP && lane == 0) {
    for (int s = 0; s < C::W_STAGES; ++s) {
      ptx::mbar_init(full_bar(s), 1);
      ptx::mbar_init(empty_bar(s), 8);  // four warps for each half
    }
    for (int s = 0; s < C::A_STAGES; ++s) {
      ptx::mbar_init(rows_bar(s), 1 + 2 * loaders);
      ptx::mbar_init(done_bar(s), 1);
    }
    for (int b = 0; b < C::BUFS; ++b) ptx::mbar_init(op_bar(b), 16);  // the same, of both CTAs
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(accf + 8u * b, 1);
      ptx::mbar_init(acce + 8u * b, 2 * C::EPI_WARPS);
      ptx::mbar_init(unitf_bar + 8u * b, 1);
      // readers of the units: epilogue, widening warps, weights' thread, rows'
      // threads and, in the leader, the MMA's
      ptx::mbar_init(unite_bar + 8u * b, C::EPI_WARPS + 8 + 1 + loaders + (rank == 0 ? 1 : 0));
    }
    ptx::mbar_init(drain_bar, 1);
    *abort_flag = 0;
    ptx::fence_barrier_init();
    ptx::prefetch_tmap(&tmA);
    if (!gather) ptx::prefetch_tmap(&tmA2);
    ptx::prefetch_tmap(&tmW1);
    if (C::FUSED) ptx::prefetch_tmap(&tmW2);
  }
  if (warp == C::MMA_WARP) {
    ptx::tmem_alloc_pair(ptx::smem_u32(tmem_slot), 512);
    ptx::tmem_relinquish_pair();
  }
  ptx::tc_fence_before();
  ptx::cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  // The kernel before this one widens the rows; its blocks let this one start once
  // they have waited for all work before them.  So everything but the widened rows
  // may be read, and Y written, without a wait for it: weights stream meanwhile.
  // SPLIT, it lets this one start at once, to set up beside the work before, which
  // for a short call is worth more: every role waits for that work (after()) before
  // its first bar, so that no clock runs meanwhile; the finder only for offsets.
  ptx::grid_launch_dependents();
  auto after = [] {
    if (C::SPLIT) ptx::grid_dependency_wait();
  };

  auto wait = [&](uint32_t bar, uint32_t parity, uint32_t where) {
    return wait_bar(bar, parity, p.timeout_ns, abort_flag, p.err, where);
  };

  // ---- epilogue (warps 0-7, both CTAs) ----
  // Warp q (mod 4) reads TMEM lanes [32q, 32q + 32), the tile's rows in the
  // columns; warps 0-3 take the even chunks of 16 rows, warps 4-7 the odd ones.
  // Linear: lane i is output column 32q + i.  FUSED: see the head of the file.
  const int q = warp & 3, h = (warp >> 2) & 1;
  const bool up = C::FUSED && (lane & 1);
  const int lcol = C::FUSED ? (lane >> 1) ^ (up ? 4 : 0) : lane;  // the lane's column in the warp's
  GroupedUnit mine = {-1, -1, 0, 0};  // the tile at hand
  bool have = false;                  // SPLIT: its sums are complete
  float w1 = 0.0f, w2 = 0.0f;
  unsigned named[3];
  float *const scales = reinterpret_cast<float *>(smem + C::SCALE_OFF + (warp & 7) * C::SCALE_BYTES);
  auto tile_col = [&](const GroupedUnit &u) {  // the warp's first column
    return (u.nb * 2 + static_cast<int>(rank)) * C::COLS + (C::FUSED ? 16 * q : 32 * q);
  };
  // The next tile's scales: of the lane's column, and of the rows of this warp's
  // chunks (16 each; lane l, word j is row l % 16 of the warp's chunk 2 j + l / 16),
  // with a bit that tells whether one names a row of A.  They are loaded while a
  // tile is finished: the two trips to memory took as long as half a tile of 1024
  // of K.
  GroupedUnit next = {-1, -1, 0, 0};
  float next_w1 = 0.0f, next_w2 = 0.0f, next_sa[3];
  int next_src[3];
  auto load_names = [&] {
    const int col = tile_col(next) + lcol;
    next_w1 = next_w2 = 0.0f;
    if (col < p.N) {
      next_w1 = ptx::load(p.s1 + int64_t(next.e) * p.N + col);
      if (C::FUSED) next_w2 = ptx::load(p.s2 + int64_t(next.e) * p.N + col);
    }
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      const int row = next.row0 + 16 * (h + 2 * (2 * j + (lane >> 4))) + (lane & 15);
      next_src[j] = -1;
      if (row < next.end) next_src[j] = p.rows ? ptx::load(p.rows + row) : row;
    }
  };
  auto load_scales = [&] {
#pragma unroll
    for (int j = 0; j < 3; ++j)
      next_sa[j] = next_src[j] >= 0 && next_src[j] < p.T ? ptx::load(p.sa + next_src[j]) : 0.0f;
  };
  auto take_scales = [&] {
    w1 = next_w1;
    w2 = next_w2;
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      scales[32 * j + lane] = next_sa[j];
      named[j] = __ballot_sync(0xffffffffu, next_src[j] >= 0 && next_src[j] < p.T);
    }
    __syncwarp();
    mine = next;
  };
  // SPLIT: the pair that finishes chunk c, and the chunk's number there.
  auto owner = [&](int c) { return (c >> 1) % p.pairs; };
  auto place = [&](int c) { return (c >> 1) / p.pairs * 2 + (c & 1); };
  // Finishes and stores the tile, whose accumulator starts at `tacc`; arrives on
  // `release` (cluster address) once the warp has read it.
  auto finish = [&](uint32_t tacc, uint32_t release) {
    const uint32_t stg = base + C::STG_OFF + warp * C::STG_BYTES;
    const int nchunk = mine.n() / 16, col0 = tile_col(mine);  // at least two chunks: one for each h
#pragma unroll 1
    for (int c = h, i = 0; c < nchunk; c += 2, ++i) {
      if (C::SPLIT && owner(c) != static_cast<int>(lead >> 1)) continue;
      uint32_t v[16];
      ptx::tmem_ld16(tacc + c * 16, v);
      ptx::tmem_wait_ld();
      ptx::reg_fence(v);
      if constexpr (C::SPLIT) {
        const float *more = reinterpret_cast<const float *>(smem) + place(c) * 16 * 128 + q * 32 + lane;
        for (int s = 1; s < p.pairs; ++s, more += C::NT / p.pairs * 128)
#pragma unroll
          for (int r = 0; r < 16; ++r) v[r] = __float_as_uint(__uint_as_float(v[r]) + more[r * 128]);
      }
      if (!C::SPLIT && c + 2 >= nchunk) {
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_cluster_relaxed(release);
      }
      const unsigned ok16 = (i < 2 ? named[0] : i < 4 ? named[1] : named[2]) >> (16 * (i & 1));
      if constexpr (C::FUSED) {
        // even lanes finish the chunk's first 8 rows, odd lanes the last 8
        const int first = up ? 8 : 0;
        const float4 sl = *reinterpret_cast<const float4 *>(scales + 16 * i + first);
        const float4 sh = *reinterpret_cast<const float4 *>(scales + 16 * i + first + 4);
        const float s[8] = {sl.x, sl.y, sl.z, sl.w, sh.x, sh.y, sh.z, sh.w};
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const uint32_t give = up ? v[r] : v[8 + r];
          const float got = __uint_as_float(__shfl_xor_sync(0xffffffffu, give, 9));
          const float mv = __uint_as_float(up ? v[8 + r] : v[r]);
          const float y = quick_silu_mul((up ? got : mv) * s[r] * w1, (up ? mv : got) * s[r] * w2);
          const __nv_bfloat16 b = __float2bfloat16_rn(y);
          // (rows 8-15 are 32 bytes further: their banks are not rows 0-7's)
          asm volatile("st.shared.b16 [%0], %1;" ::"r"(stg + (first + r) * C::STG_PITCH + first * 4 + lcol * 2),
                       "h"(*reinterpret_cast<const uint16_t *>(&b)) : "memory");
        }
      } else {
        float4 s[4];  // (loaded before any store, which they would wait for)
#pragma unroll
        for (int r = 0; r < 4; ++r) s[r] = *reinterpret_cast<const float4 *>(scales + 16 * i + 4 * r);
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const float4 &s4 = s[r / 4];
          const float sr = r % 4 == 0 ? s4.x : r % 4 == 1 ? s4.y : r % 4 == 2 ? s4.z : s4.w;
          const __nv_bfloat16 b = __float2bfloat16_rn(__uint_as_float(v[r]) * sr * w1);
          asm volatile("st.shared.b16 [%0], %1;" ::"r"(stg + r * C::STG_PITCH + lcol * 2),
                       "h"(*reinterpret_cast<const uint16_t *>(&b)) : "memory");
        }
      }
      __syncwarp();
      constexpr int PER_ROW = C::FUSED ? 2 : 4;  // 16-byte pieces
#pragma unroll
      for (int j = 0; j < PER_ROW / 2; ++j) {
        const int t = j * (32 / PER_ROW) + lane / PER_ROW, col = col0 + lane % PER_ROW * 8;
        const int row = mine.row0 + c * 16 + t;
        if (row < mine.end && col < p.N) {
          uint4 out = lds128(stg + t * C::STG_PITCH + (C::FUSED && t >= 8 ? 32 : 0) + lane % PER_ROW * 16);
          if (!((ok16 >> t) & 1u)) out = make_uint4(0, 0, 0, 0);  // no row of A
          *reinterpret_cast<uint4 *>(p.Y + int64_t(row) * p.N + col) = out;
        }
      }
      __syncwarp();
    }
  };

  if (warp < C::EPI_WARPS) {
    // ------------------------------------------------------------ epilogue
    uint32_t abuf = 0, aphase = 0;
    GroupedUnits<false> units(ring, unitf_bar, unite_bar, p.timeout_ns, p.err, abort_flag);
    after();
    bool ok = true, more = units.next(next, ok);
    if (more) {
      load_names();
      load_scales();
    }
    while (more) {
      take_scales();
      more = !C::SPLIT && units.next(next, ok);
      if (more) load_names();
      ok = __all_sync(0xffffffffu, ok && wait_bar(accf + 8u * abuf, aphase, unit_limit(p.timeout_ns, kb1 - kb0),
                                                  abort_flag, p.err, WAIT_EPI_ACC_FULL));
      if (!ok) break;
      ptx::tc_fence_after();
      if constexpr (C::SPLIT) {  // the only unit: its sums meet after the roles
        have = true;
        break;
      }
      if (more) load_scales();
      finish(tmem_base + (static_cast<uint32_t>(q * 32) << 16) + abuf * C::ACC_COLS,
             ptx::mapa_shared(acce + 8u * abuf, lead));
      if (++abuf == 2) {
        abuf = 0;
        aphase ^= 1u;
      }
    }
  } else if (warp < C::PRODUCER_WARP) {
    // ------------------------------------------------------------ weights' codes into tensor memory (both CTAs)
    // the lane's row of codes: a column of W1 or W2 (FUSED), of either half of W
    const int col = C::FUSED ? 16 * q + ((lane >> 1) ^ (lane & 1 ? 4 : 0)) : (32 * q + lane) & 63;
    const int box = C::FUSED ? lane & 1 : q >> 1;
    const uint32_t half = (warp - C::W_WARP) >> 2;
    uint32_t src[4];  // 16 codes each, in the first stage
#pragma unroll
    for (int i = 0; i < 4; ++i)
      src[i] = base + box * C::BOX_BYTES + col * C::BK + (((4 * half + i) ^ (col & 7)) << 4);
    const uint32_t dst = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + C::OP_COL + half * 32;
    uint32_t stage = 0, phase = 0, step = 0;
    bool ok = true;
    GroupedUnits<false> units(ring, unitf_bar, unite_bar, p.timeout_ns, p.err, abort_flag);
    GroupedUnit un;
    after();
    while (ok && units.next(un, ok)) {
      for (int kb = kb0; kb < kb1; ++kb, ++step) {
        const uint32_t buf = step % C::BUFS;
        ok = __all_sync(0xffffffffu, wait(full_bar(stage), phase, WAIT_MMA_FULL));
        if (!ok) break;
        uint32_t o[32];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 v = lds128(src[i] + stage * C::W_BYTES);
          widen4(v.x, o[8 * i], o[8 * i + 1]);
          widen4(v.y, o[8 * i + 2], o[8 * i + 3]);
          widen4(v.z, o[8 * i + 4], o[8 * i + 5]);
          widen4(v.w, o[8 * i + 6], o[8 * i + 7]);
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(empty_bar(stage));
        if (step >= C::BUFS) {  // the buffer's last step has been read
          const uint32_t last = step - C::BUFS;
          ok = __all_sync(0xffffffffu, wait(done_bar(last % C::A_STAGES), last / C::A_STAGES & 1u, WAIT_MMA_ACC_EMPTY));
          if (!ok) break;
          ptx::tc_fence_after();
        }
        ptx::tmem_st32(dst + buf * 64, o);
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        // (relaxed: the stores into tensor memory are complete)
        if (lane == 0) ptx::mbar_arrive_cluster_relaxed(ptx::mapa_shared(op_bar(buf), lead));
        if (++stage == C::W_STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    __syncwarp();
  } else if (warp == C::PRODUCER_WARP) {
    // ------------------------------------------------------------ copies of weights (both CTAs)
    if (ptx::elect_one()) {
      uint32_t stage = 0, phase = 0;
      bool ok = true;
      GroupedUnits<true> units(ring, unitf_bar, unite_bar, p.timeout_ns, p.err, abort_flag);
      GroupedUnit un;
      after();
      while (ok && units.next(un, ok)) {
        const int col0 = (un.nb * 2 + static_cast<int>(rank)) * C::COLS;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!(ok = wait(empty_bar(stage), phase ^ 1u, WAIT_PRODUCER_EMPTY))) break;
          const uint32_t sw = base + stage * C::W_BYTES;
          const uint32_t fb = ptx::mapa_shared(full_bar(stage), crank);
          ptx::mbar_arrive_expect_tx(full_bar(stage), C::W_BYTES);
          ptx::tma_load_3d_pair(sw, &tmW1, fb, kb * C::BK, col0, un.e);
          if (C::FUSED)
            ptx::tma_load_3d_pair(sw + C::BOX_BYTES, &tmW2, fb, kb * C::BK, col0, un.e);
          else
            ptx::tma_load_3d_pair(sw + C::BOX_BYTES, &tmW1, fb, kb * C::BK, col0 + 64, un.e);
          if (++stage == C::W_STAGES) {
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
      uint32_t step = 0, abuf = 0, aphase = 0;
      bool ok = true;
      GroupedUnits<true> units(ring, unitf_bar, unite_bar, p.timeout_ns, p.err, abort_flag);
      GroupedUnit un;
      after();
      while (ok && units.next(un, ok)) {
        const uint32_t idesc = ptx::idesc_f16(256, un.n());
        if (!(ok = wait(acce + 8u * abuf, aphase ^ 1u, WAIT_MMA_ACC_EMPTY))) break;
        ptx::tc_fence_after();
        const uint32_t d = tmem_base + abuf * C::ACC_COLS;
        for (int kb = kb0; kb < kb1; ++kb, ++step) {
          const uint32_t buf = step % C::BUFS, slot = step % C::A_STAGES;
          ok = wait(rows_bar(slot), step / C::A_STAGES & 1u, WAIT_MMA_FULL) &&
               wait(op_bar(buf), step / C::BUFS & 1u, WAIT_MMA_FULL);
          if (!ok) break;
          ptx::tc_fence_after();
          const uint32_t op = tmem_base + C::OP_COL + buf * 64;
          const uint64_t rdesc = ptx::smem_desc(base + C::A_OFF + slot * C::A_BYTES, 16, 1024, ptx::SW_128B);
          ptx::mma_f16_pair_tmem_a_k64(d, op, rdesc, idesc, kb == kb0 ? 1u : 0u);
          ptx::mma_f16_pair_tmem_a_k64(d, op + 32, rdesc + C::HALF_BYTES / 16, idesc, 0u);
          ptx::mma_commit_pair_mc(done_bar(slot), both);
        }
        if (!ok) break;
        ptx::mma_commit_pair_mc(accf + 8u * abuf, both);
        if (++abuf == 2) {
          abuf = 0;
          aphase ^= 1u;
        }
      }
      ptx::mma_commit_pair_mc(drain_bar, static_cast<uint16_t>(0x1u << lead));
      wait_quiet(drain_bar, 0, p.timeout_ns);
    }
    __syncwarp();
  } else if (warp == C::UNIT_WARP) {
    // ------------------------------------------------------------ unit finder
    if (p.offsets) after();
    find_units<C::NT, C::GROUP>(ring, off, tiles, unitf_bar, unite_bar, p.offsets, p.P, p.E, p.num_n_blk,
                                static_cast<int>(ptx::cluster_id_x()), static_cast<int>(ptx::num_clusters_x()),
                                p.timeout_ns, p.err, abort_flag);
  } else {
    // ------------------------------------------------------------ copies of rows (both CTAs)
    // As in the BF16 kernel: rows past the tile's end are not copied, and every
    // thread arrives for every step.
    const int w = warp - C::LOAD_WARP;
    if (w < loaders && ptx::elect_one()) {
      ptx::grid_dependency_wait();
      constexpr int PER = C::NT / 8 / C::LOAD_WARPS;  // gathers of a warp per step
      uint32_t step = 0;
      bool ok = true;
      GroupedUnits<true> units(ring, unitf_bar, unite_bar, p.timeout_ns, p.err, abort_flag);
      GroupedUnit un;
      while (ok && units.next(un, ok)) {
        const int row0 = un.row0 + static_cast<int>(rank) * (un.n() >> 1);
        const int rows = un.rows_of(static_cast<int>(rank));
        const uint32_t bytes = 2 * (un.row_bytes(0, gather) + un.row_bytes(1, gather));  // of both CTAs
        // the last group of four repeats the tile's last row
        int idx[PER][4];
        if (gather) {
#pragma unroll
          for (int j = 0; j < PER; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int at = min(row0 + 4 * (w + j * C::LOAD_WARPS) + i, un.end - 1);
              idx[j][i] = min(max(ptx::load(p.rows + at), 0), p.T - 1);
            }
        }
        for (int kb = kb0; kb < kb1; ++kb, ++step) {
          const uint32_t slot = step % C::A_STAGES;
          if (!(ok = wait(done_bar(slot), (step / C::A_STAGES & 1u) ^ 1u, WAIT_PRODUCER_EMPTY))) break;
          const uint32_t fb = ptx::mapa_shared(rows_bar(slot), lead);
          if (rank == 0 && w == 0) ptx::mbar_arrive_expect_tx(rows_bar(slot), bytes);
          ptx::mbar_arrive_cluster_relaxed(fb);
          const uint32_t sa = base + C::A_OFF + slot * C::A_BYTES;
          const int k = kb * C::BK;
          if (gather) {
#pragma unroll
            for (int j = 0; j < PER; ++j) {
              const int g = w + j * C::LOAD_WARPS;
              if (4 * g < rows) {
                ptx::tma_gather4_pair(sa + g * 512, &tmA, fb, k, idx[j][0], idx[j][1], idx[j][2], idx[j][3]);
                ptx::tma_gather4_pair(sa + C::HALF_BYTES + g * 512, &tmA, fb, k + 64, idx[j][0], idx[j][1], idx[j][2],
                                      idx[j][3]);
              }
            }
          } else if (rows > C::NT / 2 - 32) {
            ptx::tma_load_2d_pair(sa, &tmA2, fb, k, row0);
            ptx::tma_load_2d_pair(sa + C::HALF_BYTES, &tmA2, fb, k + 64, row0);
          } else {
            for (int i = 0; i < rows; i += 32) {
              ptx::tma_load_2d_pair(sa + i * 128, &tmA, fb, k, row0 + i);
              ptx::tma_load_2d_pair(sa + C::HALF_BYTES + i * 128, &tmA, fb, k + 64, row0 + i);
            }
          }
        }
      }
      if (!ok) {
        spin_ns(100000);  // aborted: copies already in flight into this CTA land
      } else if (w == 0) {
        // Consume the MMA's arrivals still due on this CTA's barriers, so that none
        // targets this CTA after it exits.
        for (uint32_t i = step < C::A_STAGES ? 0 : step - C::A_STAGES; i < step; ++i)
          wait_quiet(done_bar(i % C::A_STAGES), i / C::A_STAGES & 1u, p.timeout_ns);
      }
    }
    __syncwarp();
  }

  if constexpr (C::SPLIT) {
    // The pairs' sums: every copy into the rings and every MMA that reads them has
    // completed; the epilogue warps write each chunk to the pair that finishes it.
    ptx::tc_fence_before();
    __syncwarp();
    ptx::cluster_sync();
    ptx::tc_fence_after();
    const uint32_t tacc = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
    if (have) {
      const int pair = static_cast<int>(lead >> 1), nchunk = mine.n() / 16;
#pragma unroll 1
      for (int c = h; c < nchunk; c += 2) {
        const int to_pair = owner(c);
        if (to_pair == pair) continue;
        uint32_t v[16];
        ptx::tmem_ld16(tacc + c * 16, v);
        ptx::tmem_wait_ld();
        ptx::reg_fence(v);
        const int slot = pair < to_pair ? pair : pair - 1;
        const uint32_t to = ptx::mapa_shared(base, 2 * to_pair + rank) +
                            ((slot * (C::NT / p.pairs) + place(c) * 16) * 128 + q * 32 + lane) * 4;
#pragma unroll
        for (int r = 0; r < 16; ++r) ptx::st_shared_cluster_u32(to + r * 512, v[r]);
      }
    }
    __syncwarp();
    ptx::cluster_sync();
    if (have) finish(tacc, 0);
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
    ptx::tmem_dealloc_pair(tmem_base, 512);
  }
}

}  // namespace swiglu
