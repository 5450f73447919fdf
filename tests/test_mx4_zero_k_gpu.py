"""4-bit products over no values (K = 0) on the GPU: the bias, or zeros, for
rows and columns on both sides of every unit."""

import pytest
import torch

import scaled_quantize_fp8_amd as F
from tests.gpu_util import DEV
from tests.rows_util import offsets_dev

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
TILES = ["skinny16", "skinny32", "skinny48", "skinny64", "128x256", "256x256w8", None]
SIZES = [(1, 16), (1, 129), (17, 128), (65, 1), (70, 300), (130, 4096), (300, 520)]


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("M,N", SIZES)
@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("codes", [True, False])
def test_linear(monkeypatch, M, N, bias, codes, tile):
    monkeypatch.delenv("FP8L_TILE", raising=False)
    if tile is not None:
        monkeypatch.setenv("FP8L_TILE", tile)
    q, w = F.QuantizedMx4.empty(M, 0), F.QuantizedMx4.empty(N, 0)
    b = torch.arange(N, device=DEV).to(BF) if bias else None
    y = torch.full((M + 2, N), 77.0, dtype=BF, device=DEV)
    if codes:
        F.fp8_mx4_linear_fwd(q, w, b, y[1:-1])
    else:
        F.fp8_mx4_linear_fwd(torch.empty(M, 0, device=DEV), w, b, y[1:-1], q.codes, q.scale)
    want = b.expand(M, N) if bias else torch.zeros_like(y[1:-1])
    assert torch.equal(y[1:-1], want) and (y[0] == 77).all() and (y[-1] == 77).all()


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("M,N", SIZES)
@pytest.mark.parametrize("bias", [True, False])
def test_grouped(monkeypatch, M, N, bias, tile):
    monkeypatch.delenv("FP8L_TILE", raising=False)
    if tile is not None:
        monkeypatch.setenv("FP8L_TILE", tile)
    off = [1, 1 + M // 3, 1 + M // 3, 1 + M]  # rows in front, behind, and a group without any
    T = M + 3
    q, w = F.QuantizedMx4.empty(T, 0), F.QuantizedMx4.empty(3, N, 0)
    b = (torch.arange(3 * N, device=DEV) % 251).to(BF).view(3, N) if bias else None
    y = torch.full((T, N), 77.0, dtype=BF, device=DEV)
    F.fp8_mx4_grouped_linear_fwd(q, w, b, offsets_dev(off), y)
    for e in range(3):
        rows = y[off[e]:off[e + 1]]
        assert torch.equal(rows, b[e].expand_as(rows) if bias else torch.zeros_like(rows))
    assert (y[0] == 77).all() and (y[M + 1:] == 77).all()
