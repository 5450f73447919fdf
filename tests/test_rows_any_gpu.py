"""The grouped FP8 and the 8-bit integer layers on operands of any size and
alignment: odd row lengths, base pointers off every vector boundary, rows on
both sides of the tiles' edges, and every kernel that takes such operands."""

import functools

import numpy as np
import pytest
import torch

import scaled_quantize_fp8_amd as F
from oracle import fp8_oracle as O
from oracle import rows_oracle as R
from tests.gpu_util import DEV, bf16_bits, check_gemm, f32, f32_scalar, scalar_dev, to_dev, u8
from tests.rows_util import bf16, check_groups, check_i8, offsets_dev, outside, random_codes

pytestmark = pytest.mark.gpu

TILES = ["v1", "skinny16any", "skinny32any", "skinny64any", None]
# (N, K), bytes or elements that every base pointer is off: several pieces of
# K, a row shorter than a piece, aligned sizes behind unaligned pointers
SIZES = [(33, 1003, 1), (130, 4097, 3), (77, 131, 2), (64, 1040, 1), (1, 257, 0)]
OFF = [0, 17, 17, 50, 115, 116, 246]  # groups of 17, 0, 33, 65, 1, 130 rows
T = 249
SENTINEL = 7.0


def _tile(monkeypatch, tile):
    if tile is None:
        monkeypatch.delenv("FP8L_TILE", raising=False)
    else:
        monkeypatch.setenv("FP8L_TILE", tile)


def _off(t, by):
    """t on the GPU, its first element `by` elements into an allocation."""
    t = t if isinstance(t, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(t))
    buf = torch.empty(t.numel() + by, dtype=t.dtype, device=DEV)
    out = buf[by:].view(t.shape)
    out.copy_(t)
    return out


def _filled(shape, by, dtype=torch.bfloat16, value=SENTINEL):
    return _off(torch.full(shape, value, dtype=dtype), by)


@functools.lru_cache(maxsize=None)
def _fp8(N, K, fmt):
    E = len(OFF) - 1
    x8, w8 = random_codes((T, K), 1, fmt), random_codes((E, N, K), 2, fmt)
    sw = np.float32(np.random.default_rng(3).uniform(0.5, 4, E))
    b = bf16((E, N), 1.0, 9)
    return x8, w8, sw, b, R.grouped_fwd(x8, w8, fmt, np.float32(1.5), sw, OFF,
                                        f32(b).astype(float))


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("N,K,by", SIZES)
@pytest.mark.parametrize("fmt", [O.E4M3, O.E5M2])
def test_fp8_forward(N, K, by, fmt, tile, monkeypatch):
    _tile(monkeypatch, tile)
    x8, w8, sw, b, refs = _fp8(N, K, fmt)
    y = _filled((T, N), by)
    F.fp8_grouped_linear_fwd(F.Quantized(_off(x8, by), fmt, scalar_dev(1.5)),
                             F.Quantized(_off(w8, by), fmt, to_dev(sw)), _off(b, by),
                             offsets_dev(OFF), fmt, y)
    check_groups(y, refs, OFF, "y")
    assert (y.cpu()[torch.from_numpy(outside(T, OFF))] == SENTINEL).all()


@pytest.mark.parametrize("dt,hist", [(None, None), (torch.bfloat16, None), (torch.bfloat16, 16),
                                     (torch.float32, 16)])
@pytest.mark.parametrize("N,K,by", [(777, 1003, 1), (130, 515, 3), (48, 80, 1)])
def test_fp8_backward(N, K, by, dt, hist):
    """dX, dW and db from codes (dt None) or from a G quantized in the call."""
    E = len(OFF) - 1
    x8, w8 = random_codes((T, K), 1, O.E4M3), random_codes((E, N, K), 2, O.E4M3)
    g8, sg = random_codes((T, N), 5, O.E5M2), np.float32(3.0)
    dx, dw, db = _filled((T, K), by), _filled((E, N, K), by), _filled((E, N), by)
    ws = torch.empty(F.fp8_grouped_db_workspace_bytes(T, E, N), dtype=torch.uint8, device=DEV)
    codes, s = _filled((T, N), by, torch.uint8, 0xAA), torch.empty(1, device=DEV)
    if dt is None:
        g, sums = F.Quantized(_off(g8, by), O.E5M2, scalar_dev(sg)), O.dequantized(g8, O.E5M2, sg)
    else:
        G = bf16((T, N), 1e-2, 6).to(dt)
        g, sums = _off(G, by), f32(G).astype(np.float64)
        g8, sg, _ = O.quantize_step(f32(G)[:OFF[-1]], O.E5M2,
                                    None if hist is None else O.ScaleRing(hist))
    F.fp8_grouped_linear_bwd(g, O.E5M2, offsets_dev(OFF),
                             F.Quantized(_off(x8, by), O.E4M3, scalar_dev(2)),
                             F.Quantized(_off(w8, by), O.E4M3, scalar_dev(0.5)), dx, dw, db, ws,
                             None if hist is None else F.ScaleRing(hist), codes, s,
                             torch.empty(1, device=DEV))
    if dt is not None:
        assert f32_scalar(s) == np.float32(sg)
        assert np.array_equal(u8(codes)[:OFF[-1]], g8) and (u8(codes)[OFF[-1]:] == 0xAA).all()
    check_groups(dx, R.grouped_dx(g8, O.E5M2, w8, O.E4M3, sg, [np.float32(0.5)], OFF), OFF, "dx")
    assert (dx[OFF[-1]:] == SENTINEL).all()
    dbs = R.grouped_db(sums, OFF)
    for e, ref in enumerate(R.grouped_dw(g8, O.E5M2, x8, O.E4M3, sg, np.float32(2), OFF)):
        if ref is None:
            assert not dw[e].any() and not db[e].any()
        else:
            check_gemm(bf16_bits(dw[e]), ref, f"dw {e}")
            check_gemm(bf16_bits(db[e]), dbs[e], f"db {e}")


def _x(rows, K, seed):
    rng = np.random.default_rng(seed)
    return torch.from_numpy(rng.standard_normal((rows, K)) * 10.0 ** rng.uniform(-2, 2, (rows, 1))
                            ).to(torch.bfloat16)


def _weights(shape, seed=2):
    rng = np.random.default_rng(seed)
    return rng.integers(-127, 128, shape).astype(np.int8), np.float32(rng.uniform(20, 5000, shape[:-1]))


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("N,K,by", SIZES)
@pytest.mark.parametrize("M", [1, 17, 33, 65, 130])
def test_int8(M, N, K, by, tile, monkeypatch):
    _tile(monkeypatch, tile)
    out = "fp16" if M % 2 else "bf16"
    dt = torch.float16 if M % 2 else torch.bfloat16
    x, (w, sw), b = _x(M, K, 4), _weights((N, K)), bf16((N,), 2.0, 5).to(dt)
    y = _filled((M, N), by, dt)
    x8, sx = _filled((M, K), by, torch.int8), torch.empty(M, device=DEV)
    F.fp8_i8_linear_fwd(_off(x, by), F.QuantizedRows(_off(w, by), _off(sw, by)), _off(b, by), y, x8, sx)
    oq, os = R.i8_quantize_rows(f32(x))
    assert np.array_equal(x8.cpu().numpy(), oq) and np.array_equal(sx.cpu().numpy(), os)
    check_i8(y, *R.i8_linear(oq, os, w, sw, f32(b)), out)


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("N,K,by", SIZES)
def test_int8_groups(N, K, by, tile, monkeypatch):
    _tile(monkeypatch, tile)
    E = len(OFF) - 1
    x, (w, sw), b = _x(T, K, 4), _weights((E, N, K)), bf16((E, N), 2.0, 5)
    y = _filled((T, N), by)
    x8, sx = _filled((T, K), by, torch.int8, 99), torch.full((T,), -1.0, device=DEV)
    F.fp8_i8_grouped_linear_fwd(_off(x, by), F.QuantizedRows(_off(w, by), _off(sw, by)), _off(b, by),
                                offsets_dev(OFF), y, x8, sx)
    oq, os = R.i8_quantize_rows(f32(x))
    for e, i, j in R.spans(OFF):
        if i < j:
            check_i8(y[i:j], *R.i8_linear(oq[i:j], os[i:j], w[e], sw[e], f32(b)[e]), "bf16", f"group {e}")
    assert (y[OFF[-1]:] == SENTINEL).all() and (x8[OFF[-1]:] == 99).all() and (sx[OFF[-1]:] == -1).all()


@pytest.mark.parametrize("by_x,by_w", [(0, 0), (0, 1), (3, 0)])
@pytest.mark.parametrize("N,K", [(130, 1040), (77, 96)])
def test_general_tile_with_one_operand_unaligned(N, K, by_x, by_w, monkeypatch):
    """Both operands on 16-byte boundaries, or one of them off."""
    _tile(monkeypatch, "v1")
    x8, w8, sw, b, refs = _fp8(N, K, O.E4M3)
    y = _filled((T, N), 0)
    F.fp8_grouped_linear_fwd(F.Quantized(_off(x8, by_x), O.E4M3, scalar_dev(1.5)),
                             F.Quantized(_off(w8, by_w), O.E4M3, to_dev(sw)), b.to(DEV),
                             offsets_dev(OFF), O.E4M3, y)
    check_groups(y, refs, OFF, "y")
    for e in (2, 5):  # the dense layers' general tile
        i, j = OFF[e], OFF[e + 1]
        c = _filled((j - i, N), 0)
        F.fp8_gemm(F.Quantized(_off(x8[i:j], by_x), O.E4M3, scalar_dev(1.5)),
                   F.Quantized(_off(w8[e], by_w), O.E4M3, scalar_dev(sw[e])), c)
        check_gemm(bf16_bits(c), R.grouped_fwd(x8[i:j], w8[e][None], O.E4M3, np.float32(1.5),
                                               sw[e:e + 1], [0, j - i])[0], f"dense {e}")
