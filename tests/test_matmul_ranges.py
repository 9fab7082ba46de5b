"""The buffer lengths of the products' reads (csrc/mxq_matmul_ranges.hpp), compiled for
the host: no start column of a wave, past the operand's last column or not, gives a
range that ends behind the operand."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mx_microscaling_quantization_amd", "csrc")
SOURCE = """
#include "mxq_matmul_ranges.hpp"
extern "C" uint32_t operand(uint32_t rows, uint32_t C, uint32_t c0) { return mxq::operand_range(rows, C, c0); }
extern "C" uint32_t scale(uint32_t rows, uint32_t C, uint32_t c0) { return mxq::scale_range(rows, C, c0); }
"""


@pytest.fixture(scope="module")
def ranges(tmp_path_factory):
    d = tmp_path_factory.mktemp("ranges")
    (d / "ranges.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, "-o",
                    str(d / "ranges.so"), str(d / "ranges.cpp")], check=True, timeout=120)
    lib = ctypes.CDLL(str(d / "ranges.so"))
    for f in (lib.operand, lib.scale):
        f.argtypes, f.restype = [ctypes.c_uint32] * 3, ctypes.c_uint32
    return lib


# (columns, start column): one container row shorter than a wave's start, a
# remainder below 128 of a 256-column tile, the widest operand
NAMED = [(4, 64), (4, 128), (4, 192), (300, 384), (292, 384), (2880, 2944), (33554176, 33554176 + 192)]


@pytest.mark.parametrize("C,c0", NAMED)
def test_a_wave_past_the_operand_reads_nothing(ranges, C, c0):
    for rows in (1, 2, 8, 16):
        assert ranges.operand(rows, C, c0) == 0
        assert ranges.scale(rows, C, c0) == 0


def test_every_range_ends_with_the_operand(ranges):
    """Waves of 64 rows and 128 columns in tiles of 128 and 256, for every width up to
    520 containers and some wider ones."""
    for C in [*range(4, 524, 4), 2876, 2880, 2884, 33554176]:
        last_tile = (C - 1) // 256 * 256
        for c0 in [*range(0, min(C, 768) + 256, 64), last_tile, last_tile + 64, last_tile + 128, last_tile + 192]:
            for rows in (0, 1, 2, 8, 16):
                inside = c0 < C and rows > 0
                data, scale = ranges.operand(rows, C, c0), ranges.scale(rows, C, c0)
                assert data == (rows * 4 * C - 4 * c0 if inside else 0) and scale == (rows * C - c0 if inside else 0)
                assert 4 * c0 + data <= max(rows * 4 * C, 4 * c0) and c0 + scale <= max(rows * C, c0)
                assert data < 1 << 31   # a buffer's length is a positive int
