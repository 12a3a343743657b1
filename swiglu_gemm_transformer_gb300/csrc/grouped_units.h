// grouped_units.h -- how the products grouped by expert are cut into units.
// Plain arithmetic without CUDA headers: the kernel (swiglu_grouped_kernel.cuh)
// includes it for the device, the host tests for a host compiler.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define SWIGLU_UNITS_FN __device__ __forceinline__
#else
#define SWIGLU_UNITS_FN inline
#endif

namespace swiglu {

SWIGLU_UNITS_FN int units_min(int a, int b) { return a < b ? a : b; }
SWIGLU_UNITS_FN int units_max(int a, int b) { return a > b ? a : b; }

// One unit: rows [row0, end) of expert e, column tile nb; row0 = -1: no more.
// 16 bytes, read from shared memory as one int4.
struct alignas(16) GroupedUnit {
  int row0, end, e, nb;
  SWIGLU_UNITS_FN int n() const { return (end - row0 + 31) & ~31; }  // MMA N
  // Rows of the CTA `rank`'s half that belong to the tile.
  SWIGLU_UNITS_FN int rows_of(int rank) const {
    const int half = n() >> 1;
    return units_min(units_max(end - row0 - rank * half, 0), half);
  }
  // Bytes of a CTA's copies of them per stage: whole groups of four gathered
  // rows, whole boxes of dense ones.
  SWIGLU_UNITS_FN uint32_t row_bytes(int rank, bool gather) const {
    const int grain = gather ? 4 : 32;
    return ((rows_of(rank) + grain - 1) & ~(grain - 1)) * 128;
  }
};

// Units are found and handed on in blocks of this many (one per lane of a warp).
constexpr int kUnitBlock = 32;

// Time limit of the wait for a whole block of units to be taken: `limit_ns`, the
// limit of one wait, for each of them.  (Every other wait lasts about one unit at
// most: with K = 18944 a unit takes about 0.1 ms, a block 3 ms, and limits from
// 1 ms on are allowed.)  A wait that stalls ends by its own limit all the same, and
// its abort flag ends this one.
SWIGLU_UNITS_FN uint64_t block_limit(uint64_t limit_ns) {
  return limit_ns > UINT64_MAX / kUnitBlock ? UINT64_MAX : limit_ns * kUnitBlock;
}

// Sums of 32-bit places below stay below 2^31 for groups of up to 2^31 - 257
// places (the entry points refuse more): a sum that passes it would give a
// tile of a negative size.

// Row tiles of a group of `cnt` >= 0 places.
template <int NT>
SWIGLU_UNITS_FN int row_tiles(int cnt) {
  return (cnt + NT - 1) / NT;
}

// Rows of each of the `mt` tiles of a group of `cnt` >= 1 places: an even split
// in steps of 32, at most NT.  No tile is empty: cnt > (mt - 1) * NT.  (cnt +
// mt - 1 may pass 2^31, so the quotient is rounded up from cnt - 1.)
SWIGLU_UNITS_FN int tile_rows(int cnt, int mt) { return ((cnt - 1) / mt + 32) & ~31; }

// Unit u >= 0 of the call, or {-1, ...} past the last one.  off[E + 1]: the
// groups' bounds, not decreasing; tiles[E + 1]: row tiles before each group.
// Within an expert, GROUP row tiles walk the column tiles together.
template <int GROUP>
SWIGLU_UNITS_FN GroupedUnit grouped_unit(int64_t u, const int *off, const int *tiles, int E,
                                         int num_n_blk) {
  GroupedUnit r = {-1, -1, 0, 0};
  if (u >= int64_t(tiles[E]) * num_n_blk) return r;
  // the expert whose row tiles hold tile u / num_n_blk
  const int tt = static_cast<int>(u / num_n_blk);
  int lo = 0, hi = E;  // tiles[lo] <= tt < tiles[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tiles[mid] <= tt) lo = mid; else hi = mid;
  }
  const int mt = tiles[lo + 1] - tiles[lo];
  const int64_t local = u - int64_t(tiles[lo]) * num_n_blk;
  const int64_t per_group = int64_t(GROUP) * num_n_blk;
  const int first = static_cast<int>(local / per_group) * GROUP;
  const int span = units_min(GROUP, mt - first);
  const int64_t w = local % per_group;
  const int rows = tile_rows(off[lo + 1] - off[lo], mt);
  r.e = lo;
  r.nb = static_cast<int>(w / span);
  r.row0 = off[lo] + (first + static_cast<int>(w % span)) * rows;
  r.end = units_min(r.row0 + rows, off[lo + 1]);
  return r;
}

// The units of one of two warps that finish them together (they trade values
// and meet at a barrier in between).  take() is true when this warp has the next
// unit and its sums; false at the end of the units and where a wait gave up,
// which may happen to one of the two alone.  So the warps meet once for every
// take(), whatever it said: agree(ok) waits for the other warp and returns
// whether both said true.  Neither can leave while the other still waits for it.
template <class Take, class Agree, class Finish>
SWIGLU_UNITS_FN void finish_together(Take take, Agree agree, Finish finish) {
  while (agree(take())) finish();
}

}  // namespace swiglu
