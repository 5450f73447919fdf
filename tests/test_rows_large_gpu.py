"""The grouped layers on operands beyond 2^31 elements: activations, gradients
and weights whose offsets do not fit 32 bits.  A few rows hold data, the rest
are zeros, so the references stay small."""

import numpy as np
import pytest
import torch

import scaled_quantize_fp8_amd as F
from oracle import fp8_oracle as O
from oracle import rows_oracle as R
from tests.gpu_util import DEV, bf16_bits, check_gemm, f32, f32_scalar, scalar_dev, to_dev, u8
from tests.rows_util import bf16, check_i8, offsets_dev, random_codes

pytestmark = pytest.mark.gpu

WIDE, E = 8192, 3


def _rows(T):
    """(offsets, rows with data): rows at the groups' ends and past 2^31 bytes"""
    off = [0, T // 3 + 5, T // 3 + 5, T - 77]
    return off, [0, 1, off[1] - 1, off[1], off[1] + 130, off[3] - 200, off[3] - 1]


def _spread(T, width, rows, data, dtype):
    t = torch.zeros(T, width, dtype=dtype, device=DEV)
    t[torch.tensor(rows, device=DEV)] = data.to(DEV)
    return t


def _of_group(rows, off, e):
    return [i for i, r in enumerate(rows) if off[e] <= r < off[e + 1]]


def test_forward():
    T, N = 300_000, 64
    off, rows = _rows(T)
    x8, w8 = random_codes((len(rows), WIDE), 1, O.E4M3), random_codes((E, N, WIDE), 2, O.E4M3)
    y = torch.full((T, N), 7.0, dtype=torch.bfloat16, device=DEV)
    F.fp8_grouped_linear_fwd(
        F.Quantized(_spread(T, WIDE, rows, torch.from_numpy(x8), torch.uint8), O.E4M3, scalar_dev(2)),
        F.Quantized(to_dev(w8), O.E4M3, scalar_dev(0.5)), None, offsets_dev(off), O.E4M3, y)
    for e in range(E):
        at = _of_group(rows, off, e)
        if at:
            ref = O.linear_fwd(x8[at], w8[e], O.E4M3, np.float32(2), np.float32(0.5))
            check_gemm(bf16_bits(y[torch.tensor([rows[i] for i in at], device=DEV)]), ref, f"group {e}")
    y[torch.tensor(rows, device=DEV)] = 0
    assert not y[:off[-1]].any() and (y[off[-1]:] == 7).all()


# 260000 rows: one buffer resource just covers a group of them all; 300000: none does
@pytest.mark.parametrize("one_group", [False, True])
@pytest.mark.parametrize("T", [260_000, 300_000])
@pytest.mark.parametrize("hist", [None, 16])
def test_backward(T, hist, one_group):
    K = 64
    off, rows = _rows(T)
    if one_group:
        off = [0, T, T, T]
    data = bf16((len(rows), WIDE), 1e-2, 4)
    x8, w8 = random_codes((len(rows), K), 1, O.E4M3), random_codes((E, WIDE, K), 2, O.E4M3)
    g8o, sgo, ago = O.quantize_step(f32(data), O.E5M2, None if hist is None else O.ScaleRing(hist))
    G = _spread(T, WIDE, rows, data, torch.bfloat16)
    X = F.Quantized(_spread(T, K, rows, torch.from_numpy(x8), torch.uint8), O.E4M3, scalar_dev(2))
    W = F.Quantized(to_dev(w8), O.E4M3, scalar_dev(0.5))
    g8 = torch.full((T, WIDE), 0xAA, dtype=torch.uint8, device=DEV)
    dx = torch.full((T, K), 7.0, dtype=torch.bfloat16, device=DEV)
    dw, db = (torch.full(s, 7.0, dtype=torch.bfloat16, device=DEV) for s in ((E, WIDE, K), (E, WIDE)))
    ws = torch.empty(F.fp8_grouped_db_workspace_bytes(T, E, WIDE), dtype=torch.uint8, device=DEV)
    sg, ag = torch.empty(1, device=DEV), torch.empty(1, device=DEV)
    F.fp8_grouped_linear_bwd(G, O.E5M2, offsets_dev(off), X, W, dx, dw, db, ws,
                             None if hist is None else F.ScaleRing(hist), g8, sg, ag)
    at = torch.tensor(rows, device=DEV)
    assert f32_scalar(sg) == np.float32(sgo) and f32_scalar(ag) == np.float32(ago)
    assert np.array_equal(u8(g8[at]), g8o)
    g8[at] = 0
    assert not g8[:off[-1]].any() and (g8[off[-1]:] == 0xAA).all()
    for e in range(E):
        i = _of_group(rows, off, e)
        if not i:
            assert not dw[e].any() and not db[e].any()
            continue
        ref = O.linear_bwd_dx(g8o[i], O.E5M2, w8[e], O.E4M3, sgo, np.float32(0.5))
        check_gemm(bf16_bits(dx[at[i]]), ref, f"dx {e}")
        ref = O.linear_bwd_dw(g8o[i], O.E5M2, x8[i], O.E4M3, sgo, np.float32(2))
        check_gemm(bf16_bits(dw[e]), ref, f"dw {e}")
        check_gemm(bf16_bits(db[e]), O.bias_grad(f32(data)[i].astype(np.float64)), f"db {e}")
    dx[at] = 0
    assert not dx[:off[-1]].any() and (dx[off[-1]:] == 7).all()


@pytest.mark.parametrize("T", [24, 2000])
def test_weights(T):
    """40 experts of 8192 x 8192: rows of the last one, in FP8 and integers."""
    many, first = 40, 17
    off = [0] * 20 + [first] * 20 + [T]  # experts 19 and 39 have the rows
    x8 = random_codes((T, WIDE), 1, O.E4M3)
    cols = np.r_[0:64, WIDE - 64:WIDE]
    wc = {e: random_codes((len(cols), WIDE), 5 + e, O.E4M3) for e in (19, 39)}
    at = torch.from_numpy(cols).to(DEV)
    w8 = torch.zeros(many, WIDE, WIDE, dtype=torch.uint8, device=DEV)
    for e, c in wc.items():
        w8[e, at] = to_dev(c)
    y = torch.empty(T, WIDE, dtype=torch.bfloat16, device=DEV)
    F.fp8_grouped_linear_fwd(F.Quantized(to_dev(x8), O.E4M3, scalar_dev(1)),
                             F.Quantized(w8, O.E4M3, scalar_dev(1)), None, offsets_dev(off),
                             O.E4M3, y)
    for e, i, j in ((19, 0, first), (39, first, T)):
        ref = O.linear_fwd(x8[i:j], wc[e], O.E4M3, np.float32(1), np.float32(1))
        check_gemm(bf16_bits(y[i:j, at]), ref, f"expert {e}")
    y[:, at] = 0
    assert not y.any()
    q, sx = x8.view(np.int8), np.float32(np.random.default_rng(1).uniform(1, 50, T))
    sw = torch.ones(many, WIDE, device=DEV)
    F.fp8_i8_grouped_linear_fwd(F.QuantizedRows(to_dev(q), to_dev(sx)),
                                F.QuantizedRows(w8.view(torch.int8), sw), None, offsets_dev(off), y)
    for e, i, j in ((19, 0, first), (39, first, T)):
        check_i8(y[i:j, at], *R.i8_linear(q[i:j], sx[i:j], wc[e].view(np.int8),
                                          np.ones(len(cols), np.float32)), "bf16", f"expert {e}")
