"""Inputs and checks shared by the tests of the grouped and 8-bit integer
layers."""

from __future__ import annotations

import numpy as np
import torch

from oracle import fp8_oracle as O
from oracle import rows_oracle as R
from scaled_quantize_fp8_amd import workloads as WL
from tests.gpu_util import DEV, bf16_bits, check_gemm

# Row counts of the groups (then rows that belong to no group, in front and
# behind): tile edges, one row, none, more groups than a wave has lanes.
GROUPS = {
    "one": ([37], 0, 0),
    "edges": ([0, 1, 127, 128, 129, 0, 3, 255, 0], 0, 0),
    "tail": ([5, 0, 40], 0, 23),
    "front and tail": ([16, 33], 7, 9),
    "all empty": ([0, 0, 0], 0, 5),
    "few": ([20, 0, 1, 2, 16, 17] + [0, 1] * 20, 0, 3),
    "many": ([i * 7 % 5 for i in range(131)], 0, 1),
}


def offsets_of(name):
    """(T, offsets list)"""
    sizes, front, tail = GROUPS[name]
    off = [front]
    for n in sizes:
        off.append(off[-1] + n)
    return off[-1] + tail, off


def offsets_dev(off):
    return torch.tensor(off, dtype=torch.int32, device=DEV)


def random_codes(shape, seed, fmt):
    """Codes of N(0, 1) values scaled to a tenth of the format's maximum."""
    rng = np.random.default_rng(seed)
    return O.encode(np.float32(rng.standard_normal(shape) * O.fmt_max(fmt) * 0.1), fmt)


def bf16(shape, sigma, seed):
    return WL.normal_bf16(shape, sigma, seed)


def outside(T, off):
    """Mask of the rows that belong to no group."""
    m = np.ones(T, bool)
    m[off[0]:off[-1]] = False
    return m


def check_groups(out, refs, off, what):
    """Rows of a [T, n] bf16 output against per-group references."""
    bits = bf16_bits(out)
    for (e, i, j), ref in zip(R.spans(off), refs):
        if ref is not None:
            check_gemm(bits[i:j], ref, f"{what}, group {e}")


def check_i8(y, r, p, out, what=""):
    """y (torch, on the GPU) against (r, p) of rows_oracle.i8_linear."""
    got = y.detach().to("cpu").to(torch.float64).numpy()
    nan = np.isnan(r)
    assert np.array_equal(np.isnan(got), nan), f"{what}: NaN rows differ"
    if out == "fp16":  # values past the type's range round to infinity
        big = np.abs(np.where(nan, 0, r)) >= 65519
        assert not big.any(), "the case leaves fp16's range"
    bad = ~(np.abs(got - r) <= R.i8_tolerance(r, p, out)) & ~nan
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside the bound, first at "
                           f"{np.argwhere(bad)[0]}: {got[bad][0]} for {r[bad][0]}")
