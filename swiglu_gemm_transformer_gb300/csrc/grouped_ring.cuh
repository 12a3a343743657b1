// grouped_ring.cuh -- the units of the products grouped by expert (grouped_units.h)
// on the device: one warp of a CTA finds them and hands them to its other roles
// through a ring of two blocks of 32 in shared memory.
#pragma once

#include <stdint.h>

#include "grouped_units.h"
#include "sm103_ptx.cuh"
#include "tc_common.cuh"

namespace swiglu {

constexpr int kMaxExperts = 1024;

// The units of one role, in order.  Every lane of the role's warp calls
// next() (or one lane alone, for a role of one lane: ALONE).
template <bool ALONE>
class GroupedUnits {
 public:
  __device__ GroupedUnits(const GroupedUnit *ring, uint32_t full, uint32_t empty, uint64_t timeout_ns,
                          uint32_t *err, volatile int *abort_flag)
      : ring_(ring), full_(full), empty_(empty), timeout_ns_(timeout_ns), err_(err), abort_(abort_flag) {}
  // False at the end, or when a wait gave up (ok then false).
  __device__ bool next(GroupedUnit &u, bool &ok) {
    const uint32_t block = i_ >> 5;
    if ((i_ & 31u) == 0u) {
      ok = wait_bar(full_ + 8u * (block & 1u), (block >> 1) & 1u, timeout_ns_, abort_, err_,
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
  const uint64_t timeout_ns_;
  uint32_t *err_;
  volatile int *abort_;
};

// The finder's warp (every lane): the bounds and row-tile counts of the groups to
// off and tiles ([E + 1], shared), then the units cid, cid + ncl, ... to the ring.
// offsets == nullptr: one group (E = 1) of all P places.
template <int NT, int GROUP>
__device__ __forceinline__ static void find_units(GroupedUnit *ring, int *off, int *tiles, uint32_t unitf_bar,
                                                  uint32_t unite_bar, const int32_t *offsets, int P, int E,
                                                  int num_n_blk, int cid, int ncl, uint64_t timeout_ns,
                                                  uint32_t *err, volatile int *abort_flag) {
  const int lane = threadIdx.x & 31;
  // Group bounds and row-tile counts.  The bounds are clamped to [0, P] and
  // made monotone, so that no value of `offsets` reaches past Y.
  int top = 0, sum = 0;
  constexpr int AHEAD = 4;  // loads in flight: each is a trip to memory
  int raw[AHEAD];
  for (int e0 = 0; e0 <= E; e0 += 32) {
    const int e = e0 + lane, slot = (e0 / 32) % AHEAD;
    if (slot == 0) {
#pragma unroll
      for (int i = 0; i < AHEAD; ++i)
        raw[i] = e + 32 * i <= E ? (offsets ? ptx::load(offsets + e + 32 * i) : e == 0 ? 0 : P) : 0;
    }
    int v = raw[0];
#pragma unroll
    for (int i = 1; i < AHEAD; ++i) v = slot == i ? raw[i] : v;
    v = e <= E ? min(max(v, 0), P) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int w = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v = max(v, w);
    }
    v = max(v, top);
    const int prev = __shfl_up_sync(0xffffffffu, v, 1);
    // row tiles of expert e - 1
    int t = e >= 1 && e <= E ? row_tiles<NT>(v - (lane == 0 ? top : prev)) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int w = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += w;
    }
    t += sum;
    if (e <= E) {
      off[e] = v;
      tiles[e] = t;
    }
    top = __shfl_sync(0xffffffffu, v, 31);
    sum = __shfl_sync(0xffffffffu, t, 31);
  }
  __syncwarp();
  for (uint32_t block = 0;; ++block) {
    const bool ok = wait_bar(unite_bar + 8u * (block & 1u), ((block >> 1) & 1u) ^ 1u,
                             block_limit(timeout_ns), abort_flag, err, WAIT_SCHED_EMPTY);
    if (!__all_sync(0xffffffffu, ok)) break;
    const GroupedUnit r = grouped_unit<GROUP>(cid + (int64_t(block) * 32 + lane) * ncl, off,
                                                 tiles, E, num_n_blk);
    *reinterpret_cast<int4 *>(ring + 32 * (block & 1u) + lane) = make_int4(r.row0, r.end, r.e, r.nb);
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(unitf_bar + 8u * (block & 1u));
    if (__any_sync(0xffffffffu, r.row0 < 0)) break;
  }
}

}  // namespace swiglu
