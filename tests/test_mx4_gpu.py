"""Microscaled 4-bit floating point on the GPU: codes and scales bit for bit
against the oracle, exact products bit for bit, others within the bound."""

import numpy as np
import pytest
import torch

import scaled_quantize_fp8_amd as F
from oracle import mx4_oracle as X
from tests.gpu_util import DEV, f32
from tests.mx4_util import DT, check, matrix, operand

pytestmark = pytest.mark.gpu


def _quantize(x):
    q = F.QuantizedMx4.empty(*x.shape)
    q.codes.fill_(0xAB)
    q.scale.fill_(0xCD)
    F.fp8_mx4_quantize(x.to(DEV), q.codes, q.scale)
    return q


def _equal(q, x):
    c, s = X.pack(*X.quantize(f32(x)))
    assert np.array_equal(q.scale.cpu().numpy(), s), "scales differ"
    assert np.array_equal(q.codes.cpu().numpy(), c), "codes differ"


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("rows,K", [(1, 1), (1, 31), (2, 32), (3, 33), (1, 4096), (17, 127),
                                    (16, 128), (5, 129), (40, 264), (130, 72), (33, 1003), (2, 8200)])
def test_quantize_bit_exact(rows, K, dt):
    rng = np.random.default_rng(rows + K)
    x = torch.from_numpy(rng.standard_normal((rows, K)) * 10.0 ** rng.uniform(-3, 3, (rows, 1))).to(DT[dt])
    q = _quantize(x)
    _equal(q, x)
    out = torch.full((rows, K), 9.0, dtype=DT[dt], device=DEV)
    F.fp8_mx4_dequantize(q, out)
    want = X.values(*X.quantize(f32(x)))[:, :K]
    assert np.array_equal(f32(out), want)  # such values fit the inputs' type


def test_every_bf16_pattern_of_a_block():
    """Every bf16 value below 8 under the scale 1, both signs: all roundings,
    ties and saturations."""
    bits = np.arange(0x4100, dtype=np.uint16)  # 0 .. the last below 8
    bits = np.concatenate([bits, bits | 0x8000])
    bits = np.pad(bits, (0, -len(bits) % 31)).reshape(-1, 31)
    bits = np.concatenate([np.full((len(bits), 1), 0x40C0, np.uint16), bits], 1)  # 6: the scale
    x = torch.from_numpy(bits.astype(np.int16)).view(torch.bfloat16)
    _equal(_quantize(x), x)


def test_fp32_near_every_tie():
    vals = []
    for c in range(7):
        mid = np.float32((X.GRID[c] + X.GRID[c + 1]) / 2)
        vals += [mid, np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(9))]
    vals = np.float32(vals + [7.9999995, 6.5, 5.9999995] + [1e-38, 1e-45, 0.0, 3e-39])
    base = np.zeros((1, 32), np.float32)
    base[0, :len(vals)] = vals
    rows = []
    for e in range(-126, 126):
        with np.errstate(over="ignore"):
            r = base * np.float32(2.0) ** np.float32(e)
        r[0, 31] = np.float32(4.0 * 2.0 ** e) if e <= 125 else 0
        rows.append(np.where(np.isfinite(r), r, 0))
    x = torch.from_numpy(np.concatenate(rows + [-r for r in rows]))
    _equal(_quantize(x), x)


@pytest.mark.parametrize("dt", list(DT))
def test_quantize_specials(dt):
    """NaN and infinities alone in their block, zeros, subnormals, the largest."""
    x = torch.zeros(6, 160, dtype=DT[dt])
    x[0, 5], x[1, 40], x[2, 130] = float("nan"), float("inf"), -float("inf")
    x[:3, 96:100] = 1.0
    x[3] = torch.finfo(DT[dt]).max
    x[4] = torch.finfo(DT[dt]).smallest_normal / 4
    x[5, ::3] = -0.0
    q = _quantize(x)
    _equal(q, x)
    out = torch.empty(6, 160, dtype=DT[dt], device=DEV)
    F.fp8_mx4_dequantize(q, out)
    want = X.values(*X.quantize(f32(x)))
    assert np.array_equal(f32(out), want, equal_nan=True)


def test_stack_unaligned_and_empty():
    x = torch.randn(3, 5, 72, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    q = _quantize(x)
    for e in range(3):
        _equal(F.QuantizedMx4(q.codes[e], q.scale[e], 72), x[e])
    flat = torch.empty(x.numel() + 1, dtype=torch.bfloat16, device=DEV)
    xs = flat[1:].view(x.shape)
    xs.copy_(x)
    q1 = F.QuantizedMx4.empty(3, 5, 72)
    F.fp8_mx4_quantize(xs, q1.codes, q1.scale)
    assert torch.equal(q.codes, q1.codes) and torch.equal(q.scale, q1.scale)
    out = torch.empty(x.numel() + 1, dtype=torch.float32, device=DEV)[1:].view(x.shape)
    F.fp8_mx4_dequantize(q1, out)
    ref = torch.empty(x.shape, dtype=torch.float32, device=DEV)
    F.fp8_mx4_dequantize(q, ref)
    assert torch.equal(out, ref)
    for shape in ((0, 64), (4, 0), (0, 3, 8)):
        e = F.QuantizedMx4.empty(*shape)
        F.fp8_mx4_quantize(torch.empty(shape, device=DEV), e.codes, e.scale)
        F.fp8_mx4_dequantize(e, torch.empty(shape, device=DEV))


TILES = ["skinny16", "skinny32", "skinny48", "skinny64", "128x256", "256x256w8", None]
SIZES = [(1, 16, 32), (1, 1, 1), (3, 40, 96), (16, 64, 128), (17, 33, 160), (33, 77, 1003),
         (64, 130, 512), (100, 260, 288), (130, 17, 2048), (5, 300, 4100), (300, 520, 640)]


def _tile(monkeypatch, tile):
    if tile is None:
        monkeypatch.delenv("FP8L_TILE", raising=False)
    else:
        monkeypatch.setenv("FP8L_TILE", tile)


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("out", ["bf16", "fp16"])
@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_linear(monkeypatch, M, N, K, bias, out, tile):
    _tile(monkeypatch, tile)
    xc, wc = matrix(M, K, 1), matrix(N, K, 2)
    b = np.float32(np.random.default_rng(3).standard_normal(N)) if bias else None
    bt = None if b is None else torch.from_numpy(b).to(DT[out]).to(DEV)
    y = torch.full((M + 2, N), 77.0, dtype=DT[out], device=DEV)
    F.fp8_mx4_linear_fwd(operand(*xc, K), operand(*wc, K), bt, y[1:M + 1])
    r, m = X.linear(X.values(*xc), X.values(*wc), None if bt is None else f32(bt))
    check(y[1:M + 1], r, m, out)
    assert (y[0] == 77).all() and (y[-1] == 77).all()


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("M,N,K", SIZES)
def test_exact_sums(monkeypatch, M, N, K, tile):
    """Few nonzero elements of equal scales: every sum is a small multiple of a
    power of two, so the result is one rounding of the exact one."""
    _tile(monkeypatch, tile)
    rng = np.random.default_rng(M + N)
    B = -(-K // 32)
    def sparse(rows):
        c = np.zeros((rows, B, 32), np.int64)
        for r in range(rows):
            at = rng.integers(0, K, 8)
            c[r, at // 32, at % 32] = rng.integers(0, 16, 8)
        return c, np.full((rows, B), 125)
    xc, wc = sparse(M), sparse(N)
    wc[0][:, 0, 0] = rng.integers(0, 16, N)
    xc[0][:, 0, 0] = rng.integers(0, 16, M)
    y = torch.empty(M, N, dtype=torch.float16, device=DEV)
    F.fp8_mx4_linear_fwd(operand(*xc, K), operand(*wc, K), None, y)
    r, _ = X.linear(X.values(*xc), X.values(*wc))
    assert np.array_equal(f32(y), np.float32(np.float16(r)))


@pytest.mark.parametrize("tile", TILES)
def test_every_k_position_and_scale_counts(monkeypatch, tile):
    """One element of X against a W of distinct values: each position must meet
    its own element and the scales of its own block."""
    _tile(monkeypatch, tile)
    K, N = 416, 48
    rng = np.random.default_rng(5)
    B = K // 32
    xc, xe = np.zeros((K, B, 32), np.int64), np.full((K, B), 127)
    for k in range(K):
        xc[k, k // 32, k % 32] = 2  # 1.0
        xe[k, k // 32] = 120 + k % 9
    wc, we = rng.integers(0, 16, (N, B, 32)), rng.integers(122, 133, (N, B))
    y = torch.empty(K, N, dtype=torch.bfloat16, device=DEV)
    F.fp8_mx4_linear_fwd(operand(xc, xe, K), operand(wc, we, K), None, y)
    r, _ = X.linear(X.values(xc, xe), X.values(wc, we))
    assert np.array_equal(f32(y), np.float32(r))


@pytest.mark.parametrize("tile", TILES)
def test_nan_scale_stays_in_its_row(monkeypatch, tile):
    _tile(monkeypatch, tile)
    M, N, K = 37, 50, 300
    (xc, xe), (wc, we) = matrix(M, K, 1), matrix(N, K, 2)
    xe[5, 3], xc[5, 3] = 255, 0
    we[41, 9], wc[41, 9] = 255, 0
    y = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    F.fp8_mx4_linear_fwd(operand(xc, xe, K), operand(wc, we, K), None, y)
    r, m = X.linear(X.values(xc, xe), X.values(wc, we))
    check(y, r, m, "bf16")
    assert np.isnan(r).sum() == M + N - 1


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("M,N,K", SIZES)
def test_linear_quantizes_its_input(M, N, K, dt):
    wc = matrix(N, K, 2)
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(M)).to(DT[dt])
    w = operand(*wc, K)
    q = F.QuantizedMx4.empty(M, K)
    y, y2 = (torch.empty(M, N, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    F.fp8_mx4_linear_fwd(x.to(DEV), w, None, y, q.codes, q.scale)
    _equal(q, x)
    F.fp8_mx4_linear_fwd(q, w, None, y2)
    r, m = X.linear(X.values(*X.quantize(f32(x))), X.values(*wc))
    check(y, r, m, "bf16")
    check(y2, r, m, "bf16")


@pytest.mark.parametrize("tile", ["skinny16", "skinny32", "skinny48", "skinny64"])
@pytest.mark.parametrize("N,K", [(33001, 2400), (26000, 300), (12000, 1100), (4100, 7000)])
def test_few_rows_of_many_columns(monkeypatch, N, K, tile):
    """Every way of splitting K over a block's waves (none to eight); rows of W
    that repeat, so all their outputs do."""
    _tile(monkeypatch, tile)
    M = {"skinny16": 11, "skinny32": 27, "skinny48": 43, "skinny64": 59}[tile]
    wc, we = matrix(300, K, 3)
    rows = np.arange(N) % 300
    x = matrix(M, K, 4)
    y = torch.full((M, N), 7.0, dtype=torch.bfloat16, device=DEV)
    F.fp8_mx4_linear_fwd(operand(*x, K), operand(wc[rows], we[rows], K), None, y)
    r, m = X.linear(X.values(*x), X.values(wc, we))
    check(y[:, :300], r, m, "bf16")
    same = y[:, :N // 300 * 300].view(M, -1, 300)
    assert torch.equal(same, y[:, None, :300].expand_as(same))
    assert torch.equal(y[:, N // 300 * 300:], y[:, :N % 300])


def test_empty_sizes():
    w = operand(*matrix(16, 64, 1), 64)
    y = torch.empty(0, 16, dtype=torch.bfloat16, device=DEV)
    q = F.QuantizedMx4.empty(0, 64)
    F.fp8_mx4_linear_fwd(torch.empty(0, 64, device=DEV), w, None, y, q.codes, q.scale)
    k0, w0 = F.QuantizedMx4.empty(3, 0), F.QuantizedMx4.empty(8, 0)
    y = torch.full((3, 8), 9.0, dtype=torch.bfloat16, device=DEV)
    F.fp8_mx4_linear_fwd(k0, w0, None, y)
    assert not y.any()
    b = torch.arange(8, dtype=torch.bfloat16, device=DEV)
    F.fp8_mx4_linear_fwd(k0, w0, b, y)
    assert torch.equal(y, b.expand(3, 8))
