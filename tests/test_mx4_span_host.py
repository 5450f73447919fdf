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
uint32_t scale_span(int32_t steps, int32_t step, int32_t rows) {
  return fp8l::mx_scale_span(steps, step, rows);
}
int64_t piece_byte(int64_t s, int sl, int64_t K) { return fp8l::mx_piece(s, sl, K).byte; }
int64_t piece_step(int64_t s, int sl, int64_t K) { return fp8l::mx_piece(s, sl, K).step; }
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
    L.scale_span.restype = ctypes.c_uint32
    L.scale_span.argtypes = [ctypes.c_int32] * 3
    for f in (L.piece_byte, L.piece_step):
        f.restype = ctypes.c_int64
        f.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.c_int64]
    return L


@pytest.mark.parametrize("K", [0, 1, 128, 129, 300, 4096, (1 << 24) - 1])
@pytest.mark.parametrize("unit", [16, 32, 48, 64, 128])
def test_scale_descriptors_end_with_the_scales(span, unit, K):
    """Every tile of `unit` rows (of X, or columns of W) of a matrix: its
    descriptor reaches to the end of the scales at most, covers every word of
    its rows, and ends before the offset that stands for no word."""
    steps = -(-K // 128)
    for rows in (1, 3, unit - 1, unit, unit + 1, 2 * unit, 300, 1003, 4096, (1 << 29) - 1,
                 (1 << 31) - 1):
        if steps * rows >= 1 << 29:
            continue
        for first in {0, (rows - 1) // unit * unit, min(rows - 1, unit) // unit * unit}:
            here = min(unit, rows - first)
            n = span.scale_span(steps, rows, here)
            assert 0 <= n <= span.nowhere()
            assert 4 * first + n <= 4 * steps * rows or n == 0
            last = ((steps - 1) * rows + here - 1) * 4  # the last word of its rows
            assert n == (last + 4 if steps else 0)


@pytest.mark.parametrize("K", [1, 8, 31, 32, 33, 64, 72, 96, 97, 127, 128, 129, 160, 300, 513, 1003])
def test_dequantize_reads_inside_the_row(span, K):
    """Every lane of every step, up to three batches of four steps past the
    last: four bytes of the row's codes, a scale word of the row, and for a
    value of the row its own."""
    steps, row_bytes = -(-K // 128), 16 * -(-K // 32)
    for s in range(steps + 12):
        for sl in range(16):
            byte, step = span.piece_byte(s, sl, K), span.piece_step(s, sl, K)
            assert 0 <= byte <= row_bytes - 4 and 0 <= step < steps, (s, sl)
            if 128 * s + 8 * sl < K:
                assert step == s and byte == (128 * s + 8 * sl) // 2
