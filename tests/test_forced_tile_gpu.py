"""FP8L_TILE on the dense FP8 GEMMs: names of tiles that only the grouped and
integer layers have leave the dense layers' automatic choice as it is."""

import numpy as np
import pytest
import torch

import scaled_quantize_fp8_amd as F
from oracle import fp8_oracle as O
from tests.gpu_util import DEV, scalar_dev, to_dev

pytestmark = pytest.mark.gpu

M, N, K = 512, 768, 2048


def _operands():
    """Codes of every magnitude, whose products over the first half of K the
    second half takes back but for a few small ones: the rounding of the
    partial sums, and with it their order, shows in the outputs."""
    rng = np.random.default_rng(1)
    finite = np.array([c for c in range(256) if c & 0x7F != 0x7F], np.uint8)
    u, v = rng.choice(finite, (M, K // 2)), rng.choice(finite, (N, K // 2))
    small = rng.random((N, K // 2)) < 0.02
    v = np.where(small, 0x18, v).astype(np.uint8)  # 2^-4
    w = np.where(small, 0x10, v ^ 0x80).astype(np.uint8)  # 2^-5, else -v
    return np.concatenate([u, u], 1), np.concatenate([v, w], 1)


def _gemm(monkeypatch, tile):
    if tile is None:
        monkeypatch.delenv("FP8L_TILE", raising=False)
    else:
        monkeypatch.setenv("FP8L_TILE", tile)
    a, b = (F.Quantized(to_dev(c), O.E4M3, scalar_dev(1)) for c in _operands())
    c = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    F.fp8_gemm(a, b, c)
    torch.cuda.synchronize()
    return c.view(torch.int16).cpu()


@pytest.mark.parametrize("tile", ["128x256", "skinny16", "skinny32", "skinny48", "skinny64"])
def test_tiles_of_other_layers_do_not_change_the_dense_choice(tile, monkeypatch):
    """The general kernel sums in another order than the pipelined ones, so
    some of the outputs round differently: its bits show which one ran."""
    auto, general = _gemm(monkeypatch, None), _gemm(monkeypatch, "v1")
    assert not torch.equal(auto, general)
    assert torch.equal(_gemm(monkeypatch, tile), auto)
