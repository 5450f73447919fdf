"""Exchange of rows with the experts on the GPU: copies byte for byte, sums
and products within the bound that the arithmetic allows."""

import numpy as np
import pytest
import torch

import scaled_quantize_fp8_amd as F
from oracle import route_oracle as R
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25, "fp32": 2.0 ** -150}
SIZES = [(1, 1, 1), (1, 4, 64), (24, 4, 1536), (7, 8, 40), (65, 3, 129), (33, 9, 520), (5, 17, 1003), (9, 3, 9),
         (40, 2, 15), (6, 5, 7), (12, 8, 1025), (130, 2, 256), (2, 64, 8), (3, 5, 4104)]


def _places(T, k, seed):
    """Distinct places for most slots, some without one, more rows than slots."""
    rng = np.random.default_rng(seed)
    R_ = T * k + 3
    pos = rng.permutation(R_)[:T * k].reshape(T, k).astype(np.int32)
    pos[rng.random((T, k)) < 0.2] = -1
    if T > 2:
        pos[T // 2] = -1
    return R_, pos


def _rand(shape, dt, seed):
    v = np.random.default_rng(seed).standard_normal(shape)
    return torch.from_numpy(v).to(DT[dt])


def _np(t):
    return t.detach().cpu().to(torch.float64).numpy()


def _shifted(t, by):
    """The same values at an address `by` elements further."""
    flat = torch.empty(t.numel() + by, dtype=t.dtype, device=DEV)
    out = flat[by:].view(t.shape)
    out.copy_(t)
    return out


@pytest.mark.parametrize("dt", [torch.uint8, torch.bfloat16, torch.float32, torch.int64])
@pytest.mark.parametrize("T,k,D", SIZES)
@pytest.mark.parametrize("by", [0, 1])
def test_gather(T, k, D, dt, by):
    rows, pos = _places(T, k, T + D)
    rng = np.random.default_rng(D)
    as_bytes = lambda n: torch.from_numpy(rng.integers(0, 256, (n, D * dt.itemsize)).astype(np.uint8))
    x, out = as_bytes(T), as_bytes(rows)
    xd, od = (_shifted(v.to(DEV).view(dt), by) for v in (x, out))
    F.fp8_route_gather(xd, torch.from_numpy(pos).to(DEV), od)
    want = R.gather(x.numpy(), pos, out.numpy())
    assert np.array_equal(od.contiguous().view(torch.uint8).cpu().numpy(), want)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("T,k,D", SIZES)
@pytest.mark.parametrize("weighted", [True, False])
def test_combine(T, k, D, weighted, dt):
    rows, pos = _places(T, k, T + D)
    y, w = _rand((rows, D), dt, 1), np.float32(np.random.default_rng(2).random((T, k)))
    for by in (0, 1):
        out = _shifted(torch.full((T, D), 7.0, dtype=DT[dt]), by)
        F.fp8_route_combine(_shifted(y, by), torch.from_numpy(pos).to(DEV),
                            torch.from_numpy(w).to(DEV) if weighted else None, out)
        r, m = R.combine(_np(y), pos, w if weighted else None)
        d = 2.0 ** -24 * k * m  # one rounding for each fused multiply-add
        bad = ~(np.abs(_np(out) - r) <= d + HALF[dt] * (np.abs(r) + d) + TINY[dt])
        assert not bad.any()


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("T,k,D", SIZES)
def test_combine_bwd(T, k, D, dt):
    rows, pos = _places(T, k, T + D)
    y, g, old = _rand((rows, D), dt, 1), _rand((T, D), dt, 3), _rand((rows, D), dt, 4)
    w = np.float32(np.random.default_rng(2).standard_normal((T, k)))
    pd, wd = torch.from_numpy(pos).to(DEV), torch.from_numpy(w).to(DEV)
    for by in (0, 1):
        yd, gd, dy = (_shifted(v, by) for v in (y, g, old))
        dw = torch.full((T, k), 9.0, device=DEV)
        F.fp8_route_combine_bwd(gd, yd, pd, wd, dy, dw)
        rdy, rdw, mag = R.combine_bwd(_np(g), _np(y), pos, w, _np(old))
        named = np.zeros(rows, bool)
        named[pos[pos >= 0]] = True
        got = _np(dy)
        assert np.array_equal(got[~named], _np(old)[~named])
        bad = ~(np.abs(got - rdy) <= HALF[dt] * np.abs(rdy) + TINY[dt]) & named[:, None]
        assert not bad.any()
        # a term passes at most D / 64 + 8 + 6 additions of its lane and the lanes' tree
        assert (np.abs(_np(dw) - rdw) <= 2.0 ** -24 * (D / 64 + 16) * mag).all()
        # one gradient alone
        dy1, dw1 = _shifted(old, by), torch.full((T, k), 9.0, device=DEV)
        F.fp8_route_combine_bwd(gd, yd, pd, wd, None, dw1)
        F.fp8_route_combine_bwd(gd, None, pd, wd, dy1, None)
        assert torch.equal(dy1, dy) and torch.equal(dw1, dw)


def test_places_outside_the_rows_are_left_alone():
    y = _rand((4, 64), "bf16", 1).to(DEV)
    pos = torch.tensor([[0, 4], [-5, 2 ** 31 - 1], [3, -2 ** 31]], dtype=torch.int32, device=DEV)
    out = torch.full((3, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    F.fp8_route_combine(y, pos, None, out)
    assert torch.equal(out[0], y[0]) and not out[1].any() and torch.equal(out[2], y[3])
    guard = torch.full((6, 64), 5.0, dtype=torch.bfloat16, device=DEV)
    F.fp8_route_gather(out, pos, guard[1:5])
    assert (guard[0] == 5).all() and (guard[5] == 5).all() and (guard[2:4] == 5).all()
    w = torch.ones(3, 2, device=DEV)
    dw = torch.full((3, 2), 9.0, device=DEV)
    F.fp8_route_combine_bwd(out, y, pos, w, guard[1:5], dw)
    assert (guard[0] == 5).all() and (guard[5] == 5).all() and (guard[2:4] == 5).all()
    assert dw[0, 1] == 0 and not dw[1].any() and dw[2, 1] == 0


def test_the_longest_rows():
    """Rows of 2^24 - 1 bytes, and the longest sums."""
    n = (1 << 24) - 1
    x = torch.arange(n, device=DEV).to(torch.uint8).view(1, n)
    out = torch.zeros(3, n, dtype=torch.uint8, device=DEV)
    F.fp8_route_gather(x, torch.tensor([[2, 0]], dtype=torch.int32, device=DEV), out)
    assert torch.equal(out[2], x[0]) and torch.equal(out[0], x[0]) and not out[1].any()
    for D in (1 << 22, (1 << 22) - 1):
        y = torch.ones(2, D, dtype=torch.bfloat16, device=DEV)
        s = torch.empty(1, D, dtype=torch.bfloat16, device=DEV)
        pos = torch.tensor([[1, 0]], dtype=torch.int32, device=DEV)
        F.fp8_route_combine(y, pos, None, s)
        assert (s == 2).all()
        dw = torch.empty(1, 2, device=DEV)
        F.fp8_route_combine_bwd(s, y, pos, torch.ones(1, 2, device=DEV), None, dw)
        assert (dw == 2 * D).all()  # sums of whole numbers below 2^24: exact


def test_no_rows():
    e = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device=DEV)
    pos = torch.full((3, 2), -1, dtype=torch.int32, device=DEV)
    out = torch.full((3, 8), 7.0, dtype=torch.bfloat16, device=DEV)
    F.fp8_route_combine(e(0, 8), pos, None, out)
    assert not out.any()
    F.fp8_route_gather(out, pos, e(0, 8))
    dw = torch.full((3, 2), 9.0, device=DEV)
    F.fp8_route_combine_bwd(out, e(0, 8), pos, torch.ones(3, 2, device=DEV), None, dw)
    assert not dw.any()
    F.fp8_route_combine_bwd(e(3, 0), e(4, 0), pos, torch.ones(3, 2, device=DEV), None, dw.fill_(9))
    assert not dw.any()
    F.fp8_route_combine(e(4, 8), pos[:0], None, out[:0])
