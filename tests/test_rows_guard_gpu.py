"""Offsets that break the contract (decreasing, negative, past T): results are
unspecified, and no memory outside the operands is written.  Every output and
workspace lies between guard bytes that must survive."""

import pytest
import torch

import scaled_quantize_fp8_amd as F
from oracle import fp8_oracle as O
from tests.gpu_util import DEV, scalar_dev, to_dev
from tests.rows_util import bf16, offsets_dev, random_codes

pytestmark = pytest.mark.gpu

GUARD, FILL = 1 << 16, 0x5C
LOW, HIGH = -(1 << 31), (1 << 31) - 1


class Guarded:
    """Output buffers between guard bytes."""

    def __init__(self):
        self.bufs = []

    def __call__(self, *shape, dtype=torch.bfloat16):
        n = torch.empty(shape, dtype=dtype, device="meta")
        size = n.numel() * n.element_size()
        raw = torch.full((size + 2 * GUARD,), FILL, dtype=torch.uint8, device=DEV)
        self.bufs.append((raw, size))
        return raw[GUARD:GUARD + size].view(dtype).view(shape)

    def check(self):
        torch.cuda.synchronize()
        for i, (raw, size) in enumerate(self.bufs):
            assert (raw[:GUARD] == FILL).all() and (raw[GUARD + size:] == FILL).all(), f"buffer {i}"


def _offsets(kind, E, T):
    return offsets_dev({
        # more chunks of rows than the workspace holds
        "alternating": [0 if i % 2 == 0 else T for i in range(E + 1)],
        "alternating from T": [T if i % 2 == 0 else 0 for i in range(E + 1)],
        "decreasing": [T - i * T // E for i in range(E + 1)],
        "extreme": [LOW if i % 2 == 0 else HIGH for i in range(E + 1)],
        "past T": [i * T // 2 for i in range(E + 1)],
    }[kind])


KINDS = ["alternating", "alternating from T", "decreasing", "extreme", "past T"]


def _tile(monkeypatch, tile):
    if tile is None:
        monkeypatch.delenv("FP8L_TILE", raising=False)
    else:
        monkeypatch.setenv("FP8L_TILE", tile)


@pytest.mark.parametrize("tile", ["v1", "128x128w8", "256x256w8", "128x256", "skinny16", "skinny64",
                                  "skinny32any", None])
@pytest.mark.parametrize("E", [8, 130])
@pytest.mark.parametrize("kind", KINDS)
def test_forward(kind, E, tile, monkeypatch):
    _tile(monkeypatch, tile)
    T, N, K = 300, 144, 96
    out = Guarded()
    x8, y = out(T, K, dtype=torch.uint8), out(T, N)
    F.fp8_grouped_linear_fwd(bf16((T, K), 1.0, 1).to(DEV),
                             F.Quantized(to_dev(random_codes((E, N, K), 2, O.E4M3)), O.E4M3,
                                         scalar_dev(1)),
                             None, _offsets(kind, E, T), O.E4M3, y, x8_out=x8,
                             sx_used=torch.empty(1, device=DEV), amax_x=torch.empty(1, device=DEV))
    out.check()


@pytest.mark.parametrize("tile", ["v1", "128x128w8", "256x256w8", "128x256", None])
@pytest.mark.parametrize("E", [8, 130])
@pytest.mark.parametrize("N,hist", [(144, None), (272, None), (272, 16), (33, 100)])
@pytest.mark.parametrize("kind", KINDS)
def test_backward(kind, N, hist, E, tile, monkeypatch):
    _tile(monkeypatch, tile)
    T, K = 300, 96
    out = Guarded()
    g8, dx, dw, db = out(T, N, dtype=torch.uint8), out(T, K), out(E, N, K), out(E, N)
    ws = out(F.fp8_grouped_db_workspace_bytes(T, E, N), dtype=torch.uint8)
    ring = None if hist is None else F.ScaleRing(hist)
    for _ in range(1 if hist is None else 2):  # a ring's seeding call and a steady one
        F.fp8_grouped_linear_bwd(
            bf16((T, N), 1e-2, 4).to(DEV), O.E5M2, _offsets(kind, E, T),
            F.Quantized(to_dev(random_codes((T, K), 1, O.E4M3)), O.E4M3, scalar_dev(1)),
            F.Quantized(to_dev(random_codes((E, N, K), 2, O.E4M3)), O.E4M3, scalar_dev(1)), dx, dw,
            db, ws, ring, g8, torch.empty(1, device=DEV), torch.empty(1, device=DEV))
    out.check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("E", [8, 130])
def test_backward_from_codes(kind, E):
    T, N, K = 300, 144, 96
    out = Guarded()
    dx, dw, db = out(T, K), out(E, N, K), out(E, N)
    F.fp8_grouped_linear_bwd(
        F.Quantized(to_dev(random_codes((T, N), 4, O.E5M2)), O.E5M2, scalar_dev(1)), O.E5M2,
        _offsets(kind, E, T),
        F.Quantized(to_dev(random_codes((T, K), 1, O.E4M3)), O.E4M3, scalar_dev(1)),
        F.Quantized(to_dev(random_codes((E, N, K), 2, O.E4M3)), O.E4M3, scalar_dev(1)), dx, dw, db)
    out.check()


# 300 rows quantized in a launch of their own, 16 and 200 in the product's
@pytest.mark.parametrize("tile", ["v1", "128x128w8", "256x256w8", "128x256", "skinny16", "skinny64",
                                  "skinny32any", None])
@pytest.mark.parametrize("T,E", [(300, 8), (16, 8), (200, 130)])
@pytest.mark.parametrize("kind", KINDS)
def test_int8(kind, T, E, tile, monkeypatch):
    _tile(monkeypatch, tile)
    N, K = 144, 96
    out = Guarded()
    x8, sx, y = out(T, K, dtype=torch.int8), out(T, dtype=torch.float32), out(T, N)
    w = torch.randint(-127, 128, (E, N, K), dtype=torch.int8, device=DEV)
    F.fp8_i8_grouped_linear_fwd(bf16((T, K), 1.0, 1).to(DEV),
                                F.QuantizedRows(w, torch.ones(E, N, device=DEV)), None,
                                _offsets(kind, E, T), y, x8, sx)
    out.check()
