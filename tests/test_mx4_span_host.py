"""CPU checks of the offsets that the 4-bit kernels read at: the header that
holds their arithmetic, built by the host's compiler."""

import ctypes
import os
import shutil
import subprocess

import pytest

from scaled_quantize_fp8_amd import _build

SOURCE = r"""
#include "fp8l_mx4_span.hpp"
extern "C" {
uint32_t nowhere() { return fp8l::kMxNowhere; }
int64_t scale_span(int64_t steps, int64_t step, int64_t rows) {
  return fp8l::mx_scale_span(steps, step, rows);
}
}
"""


@pytest.fixture(scope="module")
def span(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("clang++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    d = tmp_path_factory.mktemp("span")
    src, so = os.path.join(d, "span.cpp"), os.path.join(d, "span.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I", _build.CSRC, src, "-o", so],
                   check=True)
    L = ctypes.CDLL(so)
    L.nowhere.restype = ctypes.c_uint32
    L.scale_span.restype = ctypes.c_int64
    L.scale_span.argtypes = [ctypes.c_int64] * 3
    return L


@pytest.mark.parametrize("K", [0, 1, 128, 129, 300, 4096, (1 << 24) - 1])
@pytest.mark.parametrize("unit", [16, 32, 48, 64, 128])
def test_scale_descriptors_end_with_the_scales(span, unit, K):
    """Every tile of `unit` rows (of X, or columns of W) of a matrix: its
    descriptor reaches to the end of the scales at most, covers every word of
    its rows, and ends before the offset that stands for no word."""
    steps = -(-K // 128)
    for rows in (1, 3, unit - 1, unit, unit + 1, 2 * unit, 300, 1003, 4096):
        if steps * rows >= 1 << 29:
            continue
        for first in {0, (rows - 1) // unit * unit, min(rows - 1, unit) // unit * unit}:
            here = min(unit, rows - first)
            n = span.scale_span(steps, rows, here)
            assert 0 <= n <= span.nowhere()
            assert 4 * first + n <= 4 * steps * rows or n == 0
            last = ((steps - 1) * rows + here - 1) * 4  # the last word of its rows
            assert n == (last + 4 if steps else 0)
