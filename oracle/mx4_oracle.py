"""Plain CPU oracle for the microscaled 4-bit floating point layers.

TEST INFRASTRUCTURE ONLY, like fp8_oracle.  numpy in 64 bits, from the
formats' definitions:

  * elements E2M1: sign, two exponent bits (bias 1), one bit of significand;
    scales E8M0: 2^(e - 127), 255 is NaN; blocks of 32 values along K;
  * a block's exponent is that of its largest magnitude less 2, at least
    2^-127; elements the nearest to x / scale, ties to the even code,
    saturating; a block with a NaN or an infinity: scale 255 and zeros;
  * matrices as the library lays them out: codes [rows, 16 B], scales
    [ceil(K / 128), rows, 4].
"""

from __future__ import annotations

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def element(code) -> float:
    """Value of a 4-bit code from its fields."""
    s, e, m = code >> 3, (code >> 1) & 3, code & 1
    mag = m * 0.5 if e == 0 else (1 + 0.5 * m) * 2.0 ** (e - 1)
    return -mag if s else mag


def nearest(v):
    """Codes (magnitude) of non-negative values: nearest, ties to even."""
    v = np.asarray(v, np.float64)
    d = np.abs(np.minimum(v, 6.0)[..., None] - GRID)
    best = d.min(-1, keepdims=True)
    tie = d == best
    # of two equally near codes the even one
    low = tie.argmax(-1)
    high = 7 - tie[..., ::-1].argmax(-1)
    return np.where(low % 2 == 0, low, high)


def exponent(amax) -> int:
    """Biased exponent of the scale of a block with this amax (not finite: NaN)."""
    if not np.isfinite(amax):
        return 255
    if amax == 0:
        return 0
    _, e = np.frexp(np.float64(amax))  # amax = f 2^e, f in [0.5, 1)
    return max(int(e) - 1 - 2 + 127, 0)


def quantize(x):
    """x [rows, K] -> (codes [rows, blocks, 32], exponents [rows, blocks])."""
    x = np.asarray(x, np.float64)
    rows, K = x.shape
    B = -(-K // 32)
    x = np.pad(x, ((0, 0), (0, B * 32 - K))).reshape(rows, B, 32)
    finite = np.isfinite(x).all(2)
    x = np.where(finite[..., None], x, 0.0)
    exps = np.vectorize(exponent, otypes=[np.int64])(np.where(finite, np.abs(x).max(2, initial=0.0), np.inf))
    scale = 2.0 ** (np.where(finite, exps, 127) - 127.0)[..., None]
    codes = nearest(np.abs(x) / scale) + 8 * np.signbit(x)
    return np.where(finite[..., None], codes, 0), exps


def values(codes, exps):
    """[rows, 32 B] values; NaN under the scale 255."""
    table = np.array([element(c) for c in range(16)])
    s = np.where(exps == 255, np.nan, 2.0 ** (np.where(exps == 255, 127, exps) - 127.0))
    return (table[codes] * s[..., None]).reshape(codes.shape[0], -1)


def pack(codes, exps):
    """The library's bytes."""
    rows, B, _ = codes.shape
    c = (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8).reshape(rows, B * 16)
    e = np.pad(exps, ((0, 0), (0, -B % 4))).astype(np.uint8)
    return c, np.ascontiguousarray(e.reshape(rows, -1, 4).transpose(1, 0, 2))


def linear(xv, wv, bias=None):
    """(r, magnitude): the unrounded result and sum of |products| of values."""
    with np.errstate(invalid="ignore"):
        r = xv @ wv.T
        m = np.abs(xv) @ np.abs(wv).T
    return (r if bias is None else r + np.asarray(bias, np.float64)), m
