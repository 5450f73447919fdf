"""Plain CPU oracle for the linear layers over ragged groups of rows and for
the row-scaled 8-bit integer layers.

TEST INFRASTRUCTURE ONLY, like fp8_oracle (whose codec and GEMM definitions
the grouped FP8 layers reuse, group by group).

  * int8 rows: s[r] = fl32(127 / max |x[r]|) and q = rint(fl32(x s)), ties to
    even; s = 1 for a row of zeros or an overflowing quotient, s = NaN and
    zeros for a row that holds a NaN or an infinity.
  * int8 linear: the integer sum is exact; y = sum / (sx sw) (+ bias), kept
    unrounded in fp64 together with the magnitude of the product part.
"""

from __future__ import annotations

import numpy as np

from . import fp8_oracle as O


def spans(offsets):
    """(group, start, end) of every group."""
    o = [int(v) for v in offsets]
    return [(e, o[e], o[e + 1]) for e in range(len(o) - 1)]


def i8_row_scale(amax) -> np.float32:
    a = np.float32(amax)
    if not np.isfinite(a):
        return np.float32(np.nan)
    if a == 0:
        return np.float32(1.0)
    with np.errstate(over="ignore"):
        s = np.float32(127.0) / a
    return s if np.isfinite(s) else np.float32(1.0)


def i8_quantize_rows(x):
    """x [rows, k] (fp32 values) -> (int8 codes, fp32 scales)."""
    x = np.asarray(x, dtype=np.float32)
    q = np.zeros(x.shape, dtype=np.int8)
    s = np.empty(x.shape[0], dtype=np.float32)
    for r in range(x.shape[0]):
        s[r] = i8_row_scale(np.max(np.abs(x[r])) if x.shape[1] else 0.0)
        if np.isfinite(s[r]):
            q[r] = np.rint(x[r] * s[r]).astype(np.int8)
    return q, s


def i8_linear(q, sx, w, sw, bias=None):
    """(r, p): the unrounded result and the product part alone, fp64."""
    acc = np.asarray(q, np.float64) @ np.asarray(w, np.float64).T  # exact: |sums| < 2^53
    with np.errstate(invalid="ignore"):
        p = acc / (np.asarray(sx, np.float64)[:, None] * np.asarray(sw, np.float64)[None])
    return (p if bias is None else p + np.asarray(bias, np.float64)), p


# Half a step of the output types, relative, and the smallest step, halved.
HALF_STEP = {"bf16": (2.0 ** -8, 2.0 ** -134), "fp16": (2.0 ** -11, 2.0 ** -25)}


def i8_tolerance(r, p, out: str):
    """Largest error of the fp32 evaluation and one rounding to `out`.

    The kernel computes fma(fl(acc), c, bias) with c = fl(fl(1/sx) fl(1/sw)):
    fl(acc) is off by at most 2^-24 relative, c by three roundings, so the
    product part p by 4 roundings (5 with their cross terms) of 2^-24, and
    the fma adds one of the result.  Then half a step of the output type."""
    half, tiny = HALF_STEP[out]
    d = 2.0 ** -24 * (5 * np.abs(p) + 2 * np.abs(r))
    return d + half * (np.abs(r) + d) + tiny


def grouped_fwd(x8, w8, fmt, sx, sw, offsets, bias=None):
    """Per group a GemmRef of its rows (None for an empty group)."""
    out = []
    for e, i, j in spans(offsets):
        b = None if bias is None else bias[e]
        out.append(None if i == j else
                   O.linear_fwd(x8[i:j], w8[e], fmt, sx, sw[e % len(sw)], b))
    return out


def grouped_dx(g8, fmt_g, w8, fmt_w, sg, sw, offsets):
    return [None if i == j else
            O.linear_bwd_dx(g8[i:j], fmt_g, w8[e], fmt_w, sg, sw[e % len(sw)])
            for e, i, j in spans(offsets)]


def grouped_dw(g8, fmt_g, x8, fmt_x, sg, sx, offsets):
    return [None if i == j else O.linear_bwd_dw(g8[i:j], fmt_g, x8[i:j], fmt_x, sg, sx)
            for e, i, j in spans(offsets)]


def grouped_db(g_values, offsets):
    return [None if i == j else O.bias_grad(g_values[i:j]) for _, i, j in spans(offsets)]
