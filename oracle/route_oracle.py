"""Plain CPU oracle for the routing to experts and the exchange of rows.

TEST INFRASTRUCTURE ONLY, like fp8_oracle.  Everything in numpy and 64 bits,
row by row, from the definitions:

  * c = p + b with p = softmax or sigmoid of the logits; groups by the sum of
    their one or two largest c; the k largest c in the groups that stay; ties
    to the lowest index; without a bias experts compare by their logits;
  * c or a logit of -inf is never chosen (index -1, weight 0); a row with a NaN
    (softmax: or +inf) takes 0 .. k-1 with NaN weights;
  * weights p, or p over the sum of the chosen, times scale, and the gradient
    of the logits with the choice held fixed;
  * a stable counting sort of the slots by expert.
"""

from __future__ import annotations

import numpy as np

SOFTMAX, SIGMOID = 0, 1
INF = np.inf


def scores(z, score):
    z = np.asarray(z, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if score == SIGMOID:
            return 1.0 / (1.0 + np.exp(-z))
        p = np.exp(z - z.max())
        return p / p.sum()


def _best(values, n):
    """Indices of the n largest, best first, ties to the lowest; -inf never."""
    order = sorted(range(len(values)), key=lambda i: (-values[i], i))[:n]
    return [i for i in order if values[i] > -INF]


def choose(z, bias, score, k, groups=1, kept=1, group_top=1):
    """The k indices of one row."""
    z = np.asarray(z, np.float64)
    E = len(z)
    bad = np.isnan(z).any() or (score == SOFTMAX and (z == INF).any())
    if bias is not None:
        bad = bad or np.isnan(bias).any()
    if bad:
        return list(range(k))
    off = z == -INF
    c = np.full(E, -INF) if off.all() else scores(z, score)
    if bias is not None:
        c = c + np.asarray(bias, np.float64)
    c = np.where(off, -INF, c)
    by = z.copy() if bias is None else c.copy()
    n = E // groups
    if groups > 1:
        of = c if group_top == 2 else by
        marks = []
        for g in range(groups):
            top = sorted((v for v in of[g * n:(g + 1) * n] if v > -INF), reverse=True)[:group_top]
            marks.append(sum(top[1:], top[0]) if top else -INF)
        stay = _best(marks, kept)
        for g in range(groups):
            if g not in stay:
                by[g * n:(g + 1) * n] = -INF
    got = _best(by, k)
    return got + [-1] * (k - len(got))


def weights(z, idx, score, renorm, scale):
    """(w, r): the weights of one row and their relative rounding bound in
    units of 2^-24 for an evaluation in 32 bits.

    Numerators exp(x): an argument off by 2^-24 |x| and an exponential off by
    two units; a sigmoid's 1 + exp(-|z|) adds four more (its exponential
    weighs at most a half) and a quotient; sums of positive terms add one unit
    for each of their at most 22 steps (16 in a lane, 6 between lanes) to the
    mean of their terms' errors; then a quotient and the scale.  Constants
    rounded up to 40 in all."""
    z = np.asarray(z, np.float64)
    live = np.array([i >= 0 for i in idx])
    zi = np.array([z[i] if i >= 0 else 0.0 for i in idx])
    if np.isnan(z).any() or (score == SOFTMAX and (z == INF).any()):
        return np.full(len(idx), np.nan), np.zeros(len(idx))
    if not live.any():
        return np.zeros(len(idx)), np.zeros(len(idx))
    with np.errstate(over="ignore"):
        if score == SIGMOID:
            low = np.minimum(zi, 0.0)
            top = low[live].max() if renorm else 0.0
            num = np.where(live, np.exp(low - top) / (1.0 + np.exp(-np.abs(zi))), 0.0)
            arg = np.abs(low - top)
        else:
            top = zi[live].max() if renorm else z.max()
            num = np.where(live, np.exp(zi - top), 0.0)
            arg = np.abs(zi - top)
    rel = np.where(live, arg, 0.0) + 40.0
    if renorm:
        q = num / num.sum()
        rel = rel + (q * np.where(live, arg, 0.0)).sum()
    elif score == SOFTMAX:
        p = scores(z, score)
        q = num / np.exp(z - top).sum()
        rel = rel + np.sum(np.where(p > 0, p * np.abs(np.where(p > 0, z, top) - top), 0.0))
    else:
        q = num
    return q * scale, rel


def gradient(z, idx, dw, score, renorm, scale):
    """(dz, bound): the gradient of one row's logits, and what an evaluation
    in 32 bits may be off, before its rounding to an output type."""
    z = np.asarray(z, np.float64)
    q, rel = weights(z, idx, score, renorm, 1.0)
    live = np.array([i >= 0 for i in idx])
    d = np.where(live, np.asarray(dw, np.float64) * scale, 0.0)
    part = q * d
    size = np.abs(part)
    top = rel.max() if len(rel) else 0.0
    if renorm:
        dot, mag = part.sum(), size.sum()
        part, size = q * (d - dot), q * (np.abs(d) + mag)
    dz, mag = np.zeros(len(z)), np.zeros(len(z))
    for i, e in enumerate(idx):
        if e < 0:
            continue
        s = 1.0
        if score == SIGMOID:
            s = 1.0 / (1.0 + np.exp(min(z[e], 700.0)))
        dz[e] += part[i] * s
        mag[e] += size[i] * s
    if score == SOFTMAX and not renorm and live.any():
        p = scores(z, score)
        dz -= p * part.sum()
        mag += p * np.abs(part).sum()
        far = np.where(p > 0, np.abs(np.where(p > 0, z, z.max()) - z.max()), 0.0)
        mag = mag * (1 + far / 64)
    # a product of two or three factors of that rounding each, a slope
    # 1 / (1 + exp(z)) off by |z| and six units, sums of at most 70 steps
    with np.errstate(invalid="ignore"):
        slope = np.abs(np.where(np.isfinite(z), z, 0.0)).max() if score == SIGMOID else 0.0
    return dz, 2.0 ** -24 * (3 * top + slope + 100) * mag


def places(idx, E):
    """(offsets [E + 1], pos of idx's shape)."""
    flat = np.asarray(idx).reshape(-1)
    pos = np.full(flat.shape, -1, np.int64)
    offsets, at = [0], 0
    for e in range(E):
        mine = np.nonzero(flat == e)[0]
        pos[mine] = at + np.arange(len(mine))
        at += len(mine)
        offsets.append(at)
    return np.array(offsets), pos.reshape(np.shape(idx))


def gather(x, pos, out):
    """out with the named rows replaced."""
    out = np.array(out)
    for t in range(pos.shape[0]):
        for p in pos[t]:
            if 0 <= p < out.shape[0]:
                out[p] = x[t]
    return out


def combine(y, pos, w):
    """(sum, sum of magnitudes) [T, D] in 64 bits."""
    T, k = pos.shape
    r, m = np.zeros((T, y.shape[1])), np.zeros((T, y.shape[1]))
    for t in range(T):
        for i in range(k):
            if 0 <= pos[t, i] < y.shape[0]:
                v = (1.0 if w is None else float(w[t, i])) * np.asarray(y[pos[t, i]], np.float64)
                r[t] += v
                m[t] += np.abs(v)
    return r, m


def combine_bwd(dout, y, pos, w, dy):
    """(dy, dw, magnitudes of dw): dy in 64 bits with the named rows replaced."""
    dy = np.array(dy, np.float64)
    T, k = pos.shape
    dw, mag = np.zeros((T, k)), np.zeros((T, k))
    g = np.asarray(dout, np.float64)
    for t in range(T):
        for i in range(k):
            p = pos[t, i]
            if 0 <= p < y.shape[0]:
                v = np.asarray(y[p], np.float64)
                dy[p] = float(w[t, i]) * g[t]
                dw[t, i] = (g[t] * v).sum()
                mag[t, i] = np.abs(g[t] * v).sum()
    return dy, dw, mag
