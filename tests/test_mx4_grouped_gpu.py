"""Experts' layers in microscaled 4-bit floating point on the GPU."""

import numpy as np
import pytest
import torch

import scaled_quantize_fp8_amd as F
from oracle import mx4_oracle as X
from tests.gpu_util import DEV, f32
from tests.mx4_util import DT, check, matrix, operand
from tests.rows_util import GROUPS, offsets_dev, offsets_of, outside

pytestmark = pytest.mark.gpu

TILES = ["skinny16", "skinny32", "skinny48", "skinny64", "128x256", "256x256w8", None]


def _weights(E, N, K):
    ms = [matrix(N, K, 10 + e) for e in range(E)]
    packed = [X.pack(*m) for m in ms]
    w = F.QuantizedMx4(*(torch.from_numpy(np.stack([p[i] for p in packed])).to(DEV)
                         for i in range(2)), K)
    return ms, w


def _check_groups(y, off, xv, ms, b, out, T):
    got = y.detach()
    for e, m in enumerate(ms):
        i, j = off[e], off[e + 1]
        if j > i:
            r, mag = X.linear(xv[i:j], X.values(*m), None if b is None else f32(b)[e])
            check(got[i:j], r, mag, out, f"group {e}")
    assert (f32(got)[outside(T, off)] == 77).all()


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("groups", list(GROUPS))
@pytest.mark.parametrize("N,K,out,bias", [(48, 160, "bf16", True), (77, 1003, "fp16", False),
                                          (272, 544, "bf16", False)])
def test_grouped(monkeypatch, groups, N, K, out, bias, tile):
    if tile is None:
        monkeypatch.delenv("FP8L_TILE", raising=False)
    else:
        monkeypatch.setenv("FP8L_TILE", tile)
    T, off = offsets_of(groups)
    E = len(off) - 1
    ms, w = _weights(E, N, K)
    b = torch.randn(E, N, generator=torch.Generator().manual_seed(1)).to(DT[out]).to(DEV) if bias else None
    xc = matrix(T, K, 5)
    y = torch.full((T, N), 77.0, dtype=DT[out], device=DEV)
    F.fp8_mx4_grouped_linear_fwd(operand(*xc, K), w, b, offsets_dev(off), y)
    _check_groups(y, off, X.values(*xc), ms, b, out, T)


@pytest.mark.parametrize("groups", list(GROUPS))
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_grouped_quantizes_rows_in_use(groups, dt):
    """Rows behind the last group, NaN here, are neither read nor written."""
    N, K = 96, 200
    T, off = offsets_of(groups)
    ms, w = _weights(len(off) - 1, N, K)
    x = torch.randn(T, K, generator=torch.Generator().manual_seed(2)).to(DT[dt])
    x[off[-1]:] = float("nan")
    q = F.QuantizedMx4.empty(T, K)
    q.codes.fill_(0xAB)
    q.scale.fill_(0xCD)
    y = torch.full((T, N), 77.0, dtype=torch.bfloat16, device=DEV)
    F.fp8_mx4_grouped_linear_fwd(x.to(DEV), w, None, offsets_dev(off), y, q.codes, q.scale)
    c, s = X.pack(*X.quantize(f32(x)))
    i, j = off[0], off[-1]
    assert np.array_equal(q.codes.cpu().numpy()[i:j], c[i:j])
    assert np.array_equal(q.scale.cpu().numpy()[:, i:j], s[:, i:j])
    assert (q.codes[j:] == 0xAB).all() and (q.scale[:, j:] == 0xCD).all()
    _check_groups(y, off, X.values(*X.quantize(np.nan_to_num(f32(x)))), ms, None, "bf16", T)
