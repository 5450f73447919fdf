"""The grouped FP8 layers on contractions long enough for every kernel's
steady loop: K, N and group sizes past 320, whole and partial last steps, odd
and even step counts, groups of more than eight tile rows."""

import functools

import numpy as np
import pytest
import torch

import scaled_quantize_fp8_amd as F
from oracle import fp8_oracle as O
from oracle import rows_oracle as R
from tests.gpu_util import DEV, bf16_bits, check_gemm, f32, scalar_dev, to_dev
from tests.rows_util import bf16, check_groups, check_i8, offsets_dev, random_codes

pytestmark = pytest.mark.gpu

OFF = [0, 300, 300, 1800, 2441, 2442, 2762]  # groups of 300, 0, 1500, 641, 1, 320 rows
T, E = 2767, 6
PIPELINED = ["128x128w8", "256x256w8", "128x256"]
SX, SG, SW = np.float32(1.5), np.float32(3.0), np.float32([0.5, 1, 2, 3, 4, 5])


def _tile(monkeypatch, tile):
    if tile is None:
        monkeypatch.delenv("FP8L_TILE", raising=False)
    else:
        monkeypatch.setenv("FP8L_TILE", tile)


@functools.lru_cache(maxsize=None)
def _operands(N, K):
    return (random_codes((T, K), 1, O.E4M3), random_codes((E, N, K), 2, O.E4M3),
            random_codes((T, N), 5, O.E5M2), bf16((E, N), 1.0, 9))


@functools.lru_cache(maxsize=None)
def _forward_refs(N, K):
    x8, w8, _, b = _operands(N, K)
    return R.grouped_fwd(x8, w8, O.E4M3, SX, SW, OFF, f32(b).astype(float))


@functools.lru_cache(maxsize=None)
def _backward_refs(N, K):
    x8, w8, g8, _ = _operands(N, K)
    return (R.grouped_dx(g8, O.E5M2, w8, O.E4M3, SG, SW, OFF),
            R.grouped_dw(g8, O.E5M2, x8, O.E4M3, SG, SX, OFF),
            R.grouped_db(O.dequantized(g8, O.E5M2, SG), OFF))


# 17.25 steps of 64 and 6.25; 5.25 and 16.25; 22 and 12
SIZES = [(400, 1104), (1040, 336), (768, 1408)]


@pytest.mark.parametrize("tile", ["v1", *PIPELINED, "skinny16", "skinny64", None])
@pytest.mark.parametrize("N,K", SIZES)
def test_forward(N, K, tile, monkeypatch):
    _tile(monkeypatch, tile)
    x8, w8, _, b = _operands(N, K)
    y = torch.empty(T, N, dtype=torch.bfloat16, device=DEV)
    F.fp8_grouped_linear_fwd(F.Quantized(to_dev(x8), O.E4M3, scalar_dev(SX)),
                             F.Quantized(to_dev(w8), O.E4M3, to_dev(SW)), b.to(DEV),
                             offsets_dev(OFF), O.E4M3, y)
    check_groups(y, _forward_refs(N, K), OFF, "y")


@pytest.mark.parametrize("tile", ["v1", *PIPELINED, None])
@pytest.mark.parametrize("N,K", SIZES)
def test_backward(N, K, tile, monkeypatch):
    """dX and dW in one launch, and in a launch each (the same tile bodies:
    the same bits)."""
    _tile(monkeypatch, tile)
    x8, w8, g8, _ = _operands(N, K)
    X, W = (F.Quantized(to_dev(x8), O.E4M3, scalar_dev(SX)),
            F.Quantized(to_dev(w8), O.E4M3, to_dev(SW)))
    G, off = F.Quantized(to_dev(g8), O.E5M2, scalar_dev(SG)), offsets_dev(OFF)
    new = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device=DEV)
    dx, dw, db = new(T, K), new(E, N, K), new(E, N)
    F.fp8_grouped_linear_bwd(G, O.E5M2, off, X, W, dx, dw, db)
    rx, rw, rb = _backward_refs(N, K)
    check_groups(dx, rx, OFF, "dx")
    for e in range(E):
        if rw[e] is None:
            assert not dw[e].any() and not db[e].any()
        else:
            check_gemm(bf16_bits(dw[e]), rw[e], f"dw {e}")
            check_gemm(bf16_bits(db[e]), rb[e], f"db {e}")
    if tile is not None:
        dx1, dw1 = new(T, K), new(E, N, K)
        F.fp8_grouped_linear_bwd(G, O.E5M2, off, None, W, dx=dx1)
        F.fp8_grouped_linear_bwd(G, O.E5M2, off, X, None, dw=dw1)
        assert torch.equal(dx1[:OFF[-1]], dx[:OFF[-1]]) and torch.equal(dw1, dw)


@pytest.mark.parametrize("tile", ["skinny16", "skinny32", "skinny48", "skinny64", "skinny16any",
                                  "skinny32any", "skinny64any", None])
@pytest.mark.parametrize("N,K", [(72, 11008), (400, 4112)])
def test_few_rows_over_a_long_contraction(N, K, tile, monkeypatch):
    """Several trips of the skinny kernels' loop over K, split over up to 8
    waves."""
    _tile(monkeypatch, tile)
    off = [0, 20, 20, 21, 23, 39, 56]
    x8, w8 = random_codes((56, K), 1, O.E4M3), random_codes((E, N, K), 2, O.E4M3)
    y = torch.empty(56, N, dtype=torch.bfloat16, device=DEV)
    F.fp8_grouped_linear_fwd(F.Quantized(to_dev(x8), O.E4M3, scalar_dev(SX)),
                             F.Quantized(to_dev(w8), O.E4M3, to_dev(SW)), None, offsets_dev(off),
                             O.E4M3, y)
    check_groups(y, R.grouped_fwd(x8, w8, O.E4M3, SX, SW, off), off, "y")


@pytest.mark.parametrize("tile", ["v1", *PIPELINED, None])
def test_int8_groups(tile, monkeypatch):
    _tile(monkeypatch, tile)
    N, K = 400, 1104
    rng = np.random.default_rng(7)
    q, w = (rng.integers(-127, 128, s).astype(np.int8) for s in ((T, K), (E, N, K)))
    sx, sw = np.float32(rng.uniform(1, 50, T)), np.float32(rng.uniform(20, 5000, (E, N)))
    y = torch.empty(T, N, dtype=torch.bfloat16, device=DEV)
    F.fp8_i8_grouped_linear_fwd(F.QuantizedRows(to_dev(q), to_dev(sx)),
                                F.QuantizedRows(to_dev(w), to_dev(sw)), None, offsets_dev(OFF), y)
    for e, i, j in R.spans(OFF):
        if i < j:
            check_i8(y[i:j], *R.i8_linear(q[i:j], sx[i:j], w[e], sw[e]), "bf16", f"group {e}")
