"""Host tests of the arithmetic that the 8-bit products are cut and timed by
(csrc/grouped_units.h, compiled here with g++): their tiles of up to 192 rows, and the
time limit of the wait for a unit's sums."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "swiglu_gemm_transformer_gb300", "csrc")

SOURCE = r"""
#include "grouped_units.h"
using namespace swiglu;
extern "C" uint64_t t_unit_limit(uint64_t ns, int steps) { return unit_limit(ns, steps); }
extern "C" int t_row_tiles(int cnt) { return row_tiles<192>(cnt); }
extern "C" int t_tile_rows(int cnt, int mt) { return tile_rows(cnt, mt); }
// out: row0, end, expert, column tile, MMA N, rows of either CTA of the units u0 .. u0 + count - 1
extern "C" void t_units(int64_t u0, int count, const int *off, const int *tiles, int E, int num_n_blk, int64_t *out) {
  for (int i = 0; i < count; ++i, out += 7) {
    const GroupedUnit u = grouped_unit<8>(u0 + i, off, tiles, E, num_n_blk);
    out[0] = u.row0, out[1] = u.end, out[2] = u.e, out[3] = u.nb, out[4] = u.n();
    out[5] = u.rows_of(0), out[6] = u.rows_of(1);
  }
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("int8_units")
    src, out = d / "units.cpp", d / "units.so"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fwrapv", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(out)], check=True)
    m = ctypes.CDLL(str(out))
    m.t_units.argtypes = [ctypes.c_int64, ctypes.c_int] + [ctypes.c_void_p] * 2 + [ctypes.c_int] * 2 + [ctypes.c_void_p]
    m.t_units.restype = None
    m.t_unit_limit.argtypes, m.t_unit_limit.restype = [ctypes.c_uint64, ctypes.c_int], ctypes.c_uint64
    return m


@pytest.mark.parametrize("ns", [10**6, 2 * 10**9, (1 << 64) - 1])
@pytest.mark.parametrize("K", [16, 1024, (1 << 17) - 16, 1 << 17, 1 << 18, (1 << 20) - 1024])
def test_limit_of_the_wait_for_a_units_sums(lib, ns, K):
    """Above what its steps take: 0.485 us each were measured, at K = 2^20 - 1024."""
    steps = -(-K // 128)
    got = lib.t_unit_limit(ns, steps)
    assert got == min(ns * (1 + steps // 1024), (1 << 64) - 1)
    assert got >= ns and got > 1.9 * 485 * steps


@pytest.mark.parametrize("cnt", [1, 31, 32, 33, 191, 192, 193, 384, 385, 700, 8191, 1 << 24, (1 << 31) - 257])
def test_tiles_of_a_group(lib, cnt):
    mt = lib.t_row_tiles(cnt)
    rows = lib.t_tile_rows(cnt, mt)
    assert mt == -(-cnt // 192) and rows % 32 == 0 and 32 <= rows <= 192
    assert (mt - 1) * rows < cnt <= mt * rows    # no tile is empty, none is missing


@pytest.mark.parametrize("num_n_blk", [1, 2, 7])
@pytest.mark.parametrize("sizes", [[0], [1], [5, 0, 3], [191, 192, 193, 0, 2], [0, 0, 4000, 0], [2999, 1, 2000, 0, 129], [31] * 70])
def test_units_take_every_place_and_column_once(lib, num_n_blk, sizes):
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    tiles = np.concatenate([[0], np.cumsum([lib.t_row_tiles(int(s)) for s in sizes])]).astype(np.int32)
    total = int(tiles[-1]) * num_n_blk
    out = np.empty((total + 3, 7), np.int64)
    lib.t_units(0, total + 3, off.ctypes.data, tiles.ctypes.data, len(sizes), num_n_blk, out.ctypes.data)
    seen = np.zeros((int(off[-1]), num_n_blk), np.int32)
    for row0, end, e, nb, n, r0, r1 in out[:total].tolist():
        assert off[e] <= row0 < end <= off[e + 1] and 32 <= n <= 192 and n % 32 == 0 and r0 + r1 == end - row0
        seen[row0:end, nb] += 1
    assert (out[total:, 0] == -1).all() and (seen == 1).all()
