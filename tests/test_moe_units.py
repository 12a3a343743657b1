"""Host tests of the arithmetic that cuts the grouped products into units
(csrc/grouped_units.h, compiled here with g++ as the kernel compiles it for the
device): every place and column once, and no sum past 32 bits up to the largest
group that the entry points accept."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "swiglu_gemm_transformer_gb300", "csrc")

SOURCE = r"""
#include <chrono>
#include <condition_variable>
#include <mutex>
#include <thread>

#include "grouped_units.h"
using namespace swiglu;
extern "C" int t_row_tiles(int nt, int cnt) { return nt == 256 ? row_tiles<256>(cnt) : row_tiles<128>(cnt); }
extern "C" uint64_t t_block_limit(uint64_t ns) { return block_limit(ns); }
extern "C" int t_tile_rows(int cnt, int mt) { return tile_rows(cnt, mt); }
// out: row0, end, expert, column tile, MMA N, rows of either CTA, bytes of either
// (dense, then gathered) of the units u0 .. u0 + count - 1
extern "C" void t_units(int64_t u0, int count, const int *off, const int *tiles, int E, int num_n_blk, int64_t *out) {
  for (int i = 0; i < count; ++i, out += 11) {
    const GroupedUnit u = grouped_unit<8>(u0 + i, off, tiles, E, num_n_blk);
    out[0] = u.row0, out[1] = u.end, out[2] = u.e, out[3] = u.nb, out[4] = u.n();
    for (int r = 0; r < 2; ++r)
      out[5 + r] = u.rows_of(r), out[7 + r] = u.row_bytes(r, false), out[9 + r] = u.row_bytes(r, true);
  }
}
// Two warps that take n[0] and n[1] units before the end (or before a wait gives
// up); done[w]: units that warp w finished.  Returns whether one of them was left
// waiting for the other.
extern "C" int t_together(const int *n, int *done) {
  std::mutex m;
  std::condition_variable cv;
  int here = 0, round = 0, stuck = 0;
  bool all = true, said = false;
  auto agree = [&](bool ok) {
    std::unique_lock<std::mutex> l(m);
    all = all && ok;
    if (++here == 2) {
      said = all, here = 0, all = true, ++round;
      cv.notify_all();
      return said;
    }
    const int mine = round;
    if (!cv.wait_for(l, std::chrono::seconds(2), [&] { return round != mine; })) {
      stuck = 1;
      return false;
    }
    return said;
  };
  auto warp = [&](int w) {
    int taken = 0;
    done[w] = 0;
    finish_together([&] { return taken++ < n[w]; }, agree, [&] { ++done[w]; });
  };
  std::thread other(warp, 1);
  warp(0);
  other.join();
  return stuck;
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("units")
    src, out = d / "units.cpp", d / "units.so"
    src.write_text(SOURCE)
    # (wrapping sums, so that one past 32 bits shows as a wrong number)
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-fwrapv", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(out)], check=True)
    m = ctypes.CDLL(str(out))
    m.t_units.argtypes = [ctypes.c_int64, ctypes.c_int] + [ctypes.c_void_p] * 2 + [ctypes.c_int] * 2 + [ctypes.c_void_p]
    m.t_units.restype = None
    m.t_block_limit.argtypes, m.t_block_limit.restype = [ctypes.c_uint64], ctypes.c_uint64
    return m


def units(lib, nt, sizes, num_n_blk, u0=0, count=None, first=0):
    off = np.concatenate([[first], first + np.cumsum(sizes, dtype=np.int64)]).astype(np.int32)
    tiles = np.concatenate([[0], np.cumsum([lib.t_row_tiles(nt, int(s)) for s in sizes])]).astype(np.int32)
    count = int(tiles[-1]) * num_n_blk + 3 if count is None else count
    out = np.empty((count, 11), np.int64)
    lib.t_units(u0, count, off.ctypes.data, tiles.ctypes.data, len(sizes), num_n_blk, out.ctypes.data)
    return off, tiles, out


LARGEST = (1 << 31) - 257   # places of one group: P stays below 2^31 - 256


@pytest.mark.parametrize("nt", [128, 256])
@pytest.mark.parametrize("cnt", [1, 31, 32, 33, 127, 128, 129, 255, 256, 257, 700, 8191, 1 << 24, (1 << 30) + 1, 2139127680,
                                 2139127681, 2139200000, (1 << 31) - 512, LARGEST - 1, LARGEST])
def test_tiles_of_a_group(lib, nt, cnt):
    mt = lib.t_row_tiles(nt, cnt)
    assert mt == -(-cnt // nt)
    rows = lib.t_tile_rows(cnt, mt)
    assert rows % 32 == 0 and 32 <= rows <= nt
    assert (mt - 1) * rows < cnt <= mt * rows    # no tile is empty, none is missing


@pytest.mark.parametrize("nt", [128, 256])
@pytest.mark.parametrize("cnt", [2139127681, 2139200000, LARGEST])
@pytest.mark.parametrize("num_n_blk", [1, 3])
def test_units_of_the_largest_groups(lib, nt, cnt, num_n_blk):
    mt = lib.t_row_tiles(nt, cnt)
    for u0 in (0, 8 * num_n_blk - 2, mt * num_n_blk // 2, mt * num_n_blk - 9 * num_n_blk, mt * num_n_blk - 2):
        _, _, out = units(lib, nt, [cnt], num_n_blk, u0, 16)
        for i, (row0, end, e, nb, n, r0, r1, d0, d1, g0, g1) in enumerate(out.tolist()):
            if u0 + i >= mt * num_n_blk:
                assert row0 == -1
                continue
            assert e == 0 and 0 <= nb < num_n_blk
            assert 0 <= row0 < end <= cnt and 32 <= n <= nt and n % 32 == 0
            assert r0 + r1 == end - row0 and r0 <= n // 2 and r1 <= n // 2
            for r, d, g in ((r0, d0, g0), (r1, d1, g1)):
                assert d == -(-r // 32) * 32 * 128 and g == -(-r // 4) * 4 * 128


@pytest.mark.parametrize("nt", [128, 256])
@pytest.mark.parametrize("num_n_blk", [1, 2, 7])
@pytest.mark.parametrize("first", [0, 5])
@pytest.mark.parametrize("sizes", [[0], [1], [5, 0, 3], [255, 256, 257, 0, 2], [0, 0, 4000, 0], [2999, 1, 2000, 0, 129], [31] * 70])
def test_units_take_every_place_and_column_once(lib, nt, num_n_blk, first, sizes):
    off, tiles, out = units(lib, nt, sizes, num_n_blk, first=first)
    seen = np.zeros((int(off[-1]), num_n_blk), np.int32)
    total = int(tiles[-1]) * num_n_blk
    for row0, end, e, nb, n, r0, r1, *_ in out[:total].tolist():
        assert off[e] <= row0 < end <= off[e + 1] and 32 <= n <= nt and r0 + r1 == end - row0
        seen[row0:end, nb] += 1
    assert (out[total:, 0] == -1).all()
    assert (seen[first:] == 1).all() and (seen[:first] == 0).all()


@pytest.mark.parametrize("n", [(0, 0), (3, 3), (0, 1), (1, 0), (2, 5), (5, 2), (64, 63), (63, 64)])
def test_two_warps_of_which_one_stops_early_both_end(lib, n):
    """One warp of two may see the end of the units (or a wait of its own give
    up) where the other does not; both leave, after the same units."""
    want, done = (ctypes.c_int * 2)(*n), (ctypes.c_int * 2)()
    assert lib.t_together(want, done) == 0
    assert list(done) == [min(n)] * 2


@pytest.mark.parametrize("ns", [10**6, 2 * 10**9, (1 << 64) // 32 - 1, (1 << 64) // 32, (1 << 64) - 1])
def test_limit_of_the_wait_for_a_block_of_units(lib, ns):
    assert lib.t_block_limit(ns) == min(32 * ns, (1 << 64) - 1)
