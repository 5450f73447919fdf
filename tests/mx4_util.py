"""Inputs and checks shared by the tests of the 4-bit floating point layers."""

from __future__ import annotations

from functools import lru_cache

import numpy as np
import torch

import scaled_quantize_fp8_amd as F
from oracle import mx4_oracle as X
from tests.gpu_util import DEV

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HALF = {"bf16": (2.0 ** -8, 2.0 ** -134), "fp16": (2.0 ** -11, 2.0 ** -25)}
# The matrix instruction's sum of a step's products keeps at least 12 bits
# below the sum of magnitudes (as for 8-bit operands, gpu_util.TIGHT_REL).
SUM_REL = 2.0 ** -10


@lru_cache(maxsize=None)
def _matrix(rows, K, seed, spread=2.0):
    """Codes and exponents of a matrix whose rows' sizes differ."""
    rng = np.random.default_rng(seed)
    v = rng.standard_normal((rows, K)) * 2.0 ** rng.uniform(-spread, spread, (rows, 1))
    return X.quantize(np.float32(v))


def matrix(rows, K, seed, spread=2.0):
    return tuple(a.copy() for a in _matrix(rows, K, seed, spread))


def operand(codes, exps, K):
    c, s = X.pack(codes, exps)
    return F.QuantizedMx4(torch.from_numpy(c).to(DEV), torch.from_numpy(s).to(DEV), K)


def check(y, r, m, out, what=""):
    """y (torch) against the unrounded results r and sums of magnitudes m."""
    got = y.detach().cpu().to(torch.float64).numpy()
    nan = np.isnan(r)
    assert np.array_equal(np.isnan(got), nan), f"{what}: NaN outputs differ"
    half, tiny = HALF[out]
    d = SUM_REL * m + 2.0 ** -24 * np.abs(r)  # the sums, the bias' addition
    bad = ~(np.abs(got - r) <= d + half * (np.abs(r) + d) + tiny) & ~nan
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside the bound, first at "
                           f"{np.argwhere(bad)[0]}: {got[bad][0]} for {r[bad][0]}")
