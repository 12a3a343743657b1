"""Host tests of how the routers' one-launch form shares its tokens out
(csrc/route_blocks.h, compiled here with g++)."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "swiglu_gemm_transformer_gb300", "csrc")

SOURCE = r"""
#include "route_blocks.h"
using namespace swiglu;
static OneLaunch how(int lanes, int per_lane) { return per_lane ? one_by_score(per_lane & 63, per_lane & 64 ? 32 : 8) : one_by_logit(lanes); }
extern "C" int t_tokens(int T, int lanes, int per_lane) { return one_block_tokens(T, how(lanes, per_lane)); }
extern "C" int t_blocks(int T, int lanes, int per_lane) { return one_blocks(T, t_tokens(T, lanes, per_lane)); }
"""

LONG = 64   # 32 choices a token instead of 8
FORMS = [(4, 0), (8, 0), (16, 0), (32, 0), (32, 2), (32, 8), (32, 16), (32, 32), (32, 8 + LONG)]   # lanes of a token; by scores: experts of a lane


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("blocks")
    src, out = d / "blocks.cpp", d / "blocks.so"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(out)], check=True)
    return ctypes.CDLL(str(out))


@pytest.mark.parametrize("form", FORMS, ids=str)
def test_every_token_has_a_block(lib, form):
    for T in range(1, 257):
        tokens, blocks = lib.t_tokens(T, *form), lib.t_blocks(T, *form)
        assert 1 <= blocks <= 8 and blocks & (blocks - 1) == 0
        assert tokens * blocks >= T and 1 <= tokens <= 32


# Tokens at which one block was measured at least 3 % faster than several, and the other way round.
@pytest.mark.parametrize("form,alone,shared", [((8, 0), (9, 12, 16, 20, 24), (33, 40, 64)), ((4, 0), (9, 16, 24, 32), (64,)),
                                               ((16, 0), (9, 12, 16), (26, 32, 64)), ((32, 0), (9, 10, 12), (16, 24, 64)),
                                               ((32, 2), (9, 12, 16), (24, 32, 64)), ((32, 8), (9, 12), (17, 24, 64)),
                                               ((32, 32), (9, 12), (16, 24, 64)), ((32, 8 + LONG), (1, 8), (13, 15, 32))], ids=str)
def test_small_calls_take_the_faster_form(lib, form, alone, shared):
    for T in alone:
        assert lib.t_blocks(T, *form) == 1
    for T in shared:
        assert lib.t_blocks(T, *form) > 1
