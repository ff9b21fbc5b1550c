"""The 4-bit product's choice of kernel: host code, compiled here by itself.  It takes what was
fastest where all kernels were measured, and sends the sizes of the GPU tests to the kernels that
they are meant for."""
from __future__ import annotations

import ctypes
import os
import subprocess

import pytest

from tests import test_gpu_mx4_tiles as tiles

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "w8a8_int8_quantized_qk_amd", "csrc")
NAMES = ["16x64", "16x32", "16x16", "32x32 few", "32x16 few", "rows 32", "rows 64", "128x128", "128x256", "256x256"]


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    where = tmp_path_factory.mktemp("rule")
    (where / "rule.cpp").write_text('#include "mx4_rule.h"\nextern "C" int kernel_of(int m, int n, int k) '
                                    '{ return static_cast<int>(qk::mx4_kernel_of(m, n, k)); }\n')
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, str(where / "rule.cpp"),
                    "-o", str(where / "rule.so")], check=True)
    lib = ctypes.CDLL(str(where / "rule.so"))
    return lambda m, n, k: NAMES[lib.kernel_of(m, n, k)]


# us of rows 64 / 128x128 / 128x256 / 256x256, two operands in turn (None: not measured, far slower)
MEASURED = {
    (256, 4096, 14336): (22.5, 32.0, 53.9, None), (512, 4096, 14336): (39.6, 32.3, 53.9, None), (1024, 4096, 14336): (None, 37.9, 54.1, None),
    (1500, 4096, 14336): (None, 64.9, 55.2, 74.8), (2048, 4096, 14336): (None, 74.1, 61.3, 74.8), (3000, 4096, 14336): (None, 110.4, 111.6, 84.8),
    (4096, 4096, 14336): (None, 141.3, 123.4, 98.6), (6000, 4096, 14336): (None, 212.8, 183.8, 169.9),
    (1024, 6144, 14336): (None, 65.9, 55.2, 75.0), (2048, 6144, 14336): (None, 106.0, 111.6, 83.2), (4096, 6144, 14336): (None, 221.2, 184.6, 170.0),
    (768, 14336, 14336): (None, 103.2, 118.9, 80.7), (512, 4096, 4096): (18.4, 13.1, 19.2, None), (1024, 4096, 4096): (None, 13.8, 19.5, None),
    (1500, 4096, 4096): (47.8, 25.1, 20.1, 27.2), (2048, 4096, 4096): (None, 26.2, 21.6, 27.3), (3000, 4096, 4096): (None, 38.8, 39.0, 29.2),
    (4096, 4096, 4096): (None, 50.0, 42.4, 34.8), (768, 14336, 4096): (None, 37.3, 39.2, 27.7), (2048, 6144, 4096): (None, 38.3, 39.1, 29.3),
    (6000, 6144, 4096): (None, 110.9, 98.7, 90.7), (1024, 1024, 4096): (11.3, 12.7, 17.3, None), (4096, 1024, 4096): (None, 13.8, 19.6, None),
    (3000, 6144, 1024): (58.5, 31.1, 25.3, 24.9), (2048, 1024, 1024): (8.3, 7.2, 8.8, 12.1), (4096, 14336, 1024): (None, 88.9, 60.4, 51.2)}


@pytest.mark.parametrize("size", MEASURED, ids=lambda s: "x".join(map(str, s)))
def test_the_fastest_is_taken(rule, size):
    times = dict(zip(NAMES[6:], MEASURED[size]))
    taken, best = times.get(rule(*size)), min(t for t in times.values() if t)
    assert taken is not None and taken <= 1.04 * best, (rule(*size), times)


def test_sizes_of_the_tiles_tests(rule):
    assert [rule(*s) for s in tiles.SIZES] == ["128x128"] * 3 + ["128x256"] * 3 + ["256x256"] * 3
    for k in (992, 1024, 2048, 2176, 4352):
        assert [rule(m, n, k) for m, n in ((700, 4096), (2000, 4000), (3100, 4096))] == NAMES[7:]


@pytest.mark.parametrize("m,n,k,want", [(1, 25600, 4096, "16x64"), (16, 25599, 4096, "16x32"), (1, 12799, 32, "16x16"), (17, 12800, 64, "32x32 few"),
                                        (32, 12799, 64, "32x16 few"), (33, 300, 4096, "rows 32"), (200, 4096, 4096, "rows 64"),
                                        (1 << 24, 1 << 24, 32, "rows 64"), (1 << 24, 1 << 24, 1 << 24, "256x256"), (33, 1, 0, "rows 32")])
def test_ends_of_the_range(rule, m, n, k, want):
    assert rule(m, n, k) == want
