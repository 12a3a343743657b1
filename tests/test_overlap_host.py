"""Kernels that start while earlier work of their stream still runs read what that work
may write with ordinary loads (no GPU: the sources are read).

The read-only path (__ldg, ld.global.nc, const __restrict__ arguments) is for memory
that nothing writes during a kernel's whole life.  A kernel of a programmatic launch
lives before the kernels in front of it have written their outputs, which are its inputs."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "swiglu_gemm_transformer_gb300", "csrc")

# Launched in order, after all earlier work (repacking of weights), or reading only what
# was complete before the first launch of their call, an ordered one (the FP8 producer).
IN_ORDER = {"k_misc.cu", "k_fp8.cu", "k_dqt.cu", "k_producer.cu"}
READ_ONLY_PATH = re.compile(r"__ldg\s*\(|\.nc\b|const\s+\w+\s*\*\s*__restrict__")


def sources():
    return sorted(os.path.basename(f) for p in ("*.cu", "*.cuh") for f in glob.glob(os.path.join(CSRC, p)))


def code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", [n for n in sources() if n not in IN_ORDER])
def test_overlapped_kernels_keep_off_the_read_only_path(name):
    found = [m.group(0) for m in READ_ONLY_PATH.finditer(code(name))]
    assert not found, f"{name}: {found}"


@pytest.mark.parametrize("name", sorted(IN_ORDER - {"k_producer.cu"}))
def test_kernels_on_the_read_only_path_are_launched_in_order(name):
    text, seen = code(name), 0
    for part in text.split("__global__")[1:]:
        kernel = re.match(r"\s*void\s+(?:__launch_bounds__\([^)]*\)\s*)?(\w+)\s*\(", part).group(1)
        if READ_ONLY_PATH.search(part[:part.index("\n}\n")]):
            assert kernel + "<<<" in text, kernel
            seen += 1
    assert seen > 0
