"""Routing, exchange and 4-bit layers over arrays of more than 2^31 elements
or bytes, and guard bytes around every output."""

import numpy as np
import pytest
import torch

import scaled_quantize_fp8_amd as F
from oracle import mx4_oracle as X
from oracle import route_oracle as R
from tests.gpu_util import DEV, f32
from tests.mx4_util import check, matrix, operand
from tests.rows_util import bf16, offsets_dev

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _ends(n):
    return [0, 1, n // 2, n - 2, n - 1]


def test_route_of_many_logits():
    """2.2 million tokens of 1000 experts: forward, places and gradient."""
    T, E, k = 2_200_000, 1000, 1
    z = torch.zeros(T, E, dtype=BF, device=DEV)
    best = (torch.arange(T, device=DEV) * 7919 % E).to(torch.int32)
    z.scatter_(1, best.long()[:, None], 3.0)
    idx, pos = (torch.empty(T, k, dtype=torch.int32, device=DEV) for _ in range(2))
    w, off = torch.empty(T, k, device=DEV), torch.empty(E + 1, dtype=torch.int32, device=DEV)
    ws = torch.empty(F.fp8_route_workspace_bytes(T, E, k), dtype=torch.uint8, device=DEV)
    F.fp8_route_fwd(z, idx, w, renorm=False, offsets=off, pos=pos, ws=ws)
    assert torch.equal(idx[:, 0], best)
    count = torch.bincount(best.long(), minlength=E)
    assert torch.equal(off[1:].long(), count.cumsum(0)) and int(off[0]) == 0
    order = best.long().argsort(dim=0, stable=True)
    assert torch.equal(pos.view(-1)[order].long(), torch.arange(T, device=DEV))
    p = np.exp(3.0) / (np.exp(3.0) + E - 1)
    assert ((w.double() - p).abs() <= 2.0 ** -24 * 64 * p).all()
    dz = torch.empty_like(z)
    F.fp8_route_bwd(z, idx, torch.ones_like(w), dz, renorm=False)
    for t in _ends(T):
        r, d = R.gradient(f32(z[t]).astype(np.float64), [int(best[t])], np.ones(1), 0, False, 1.0)
        tol = d + 2.0 ** -8 * (np.abs(r) + d)
        assert (np.abs(f32(dz[t]) - r) <= tol).all(), t


def test_exchange_of_many_elements():
    """Rows whose elements pass 2^31, in and out."""
    T, k, D = 140_000, 2, 16_384
    x = torch.zeros(T, D, dtype=BF, device=DEV)
    at = torch.tensor(_ends(T), device=DEV)
    x[at] = torch.randn(5, D, device=DEV).to(BF)
    pos = torch.arange(T * k, dtype=torch.int32, device=DEV).view(T, k).flip(0)
    xs = torch.full((T * k, D), 3.0, dtype=BF, device=DEV)
    F.fp8_route_gather(x, pos, xs)
    for i in range(k):
        assert torch.equal(xs[pos[at, i].long()], x[at])
    w = torch.full((T, k), 0.5, device=DEV)
    out = torch.full((T, D), 3.0, dtype=BF, device=DEV)
    F.fp8_route_combine(xs, pos, w, out)
    assert torch.equal(out, x)  # halves of the same value, twice
    dw, dy = torch.empty(T, k, device=DEV), torch.full_like(xs, 3.0)
    F.fp8_route_combine_bwd(x, xs, pos, w, dy, dw)
    want = (x[at].double() ** 2).sum(1)
    assert ((dw[at].double() - want[:, None]).abs() <= 2.0 ** -24 * (D / 64 + 16) * want[:, None]).all()
    for i in range(k):
        assert torch.equal(dy[pos[at, i].long()], (x[at].float() * 0.5).to(BF))
    rest = torch.ones(T, dtype=torch.bool, device=DEV)
    rest[at] = False
    assert not dw[rest].any()


def test_quantize_many_elements():
    rows, K = 140_000, 16_400
    x = torch.zeros(rows, K, dtype=BF, device=DEV)
    at = _ends(rows)
    x[torch.tensor(at, device=DEV)] = torch.randn(5, K, device=DEV).to(BF)
    q = F.QuantizedMx4.empty(rows, K)
    F.fp8_mx4_quantize(x, q.codes, q.scale)
    back = torch.full((rows, K), 3.0, dtype=BF, device=DEV)
    F.fp8_mx4_dequantize(q, back)
    for t in at:
        v = X.values(*X.quantize(f32(x[t:t + 1])))
        assert np.array_equal(f32(back[t:t + 1]), np.float32(v[:, :K]))
    assert not back[2:rows // 2].any() and not back[rows // 2 + 1:rows - 2].any()


@pytest.mark.parametrize("grouped", [False, True])
def test_linear_of_many_rows(grouped):
    """X codes of more than 2^31 bytes, and Y of more than 2^31 elements."""
    for M, N, K in ((150_000, 64, 32_000), (600_000, 4096, 64)):
        w = matrix(N, K, 3)
        xr = matrix(5, K, 4)
        q = F.QuantizedMx4.empty(M, K)
        q.codes.zero_()
        q.scale.fill_(127)
        at = torch.tensor(_ends(M), device=DEV)
        few = operand(*xr, K)
        q.codes[at] = few.codes
        q.scale[:, at] = few.scale
        y = torch.full((M, N), 7.0, dtype=BF, device=DEV)
        W = operand(*w, K)
        if grouped:
            W = F.QuantizedMx4(W.codes[None], W.scale[None], K)
            F.fp8_mx4_grouped_linear_fwd(q, W, None, offsets_dev([0, M]), y)
        else:
            F.fp8_mx4_linear_fwd(q, W, None, y)
        r, m = X.linear(X.values(*xr), X.values(*w))
        check(y[at], r, m, "bf16", f"{M}")
        assert not y[2:M // 2].any() and not y[M // 2 + 1:M - 2].any()


def test_weights_of_many_experts():
    """Expert weights of more than 2^32 bytes of codes: the last experts'."""
    E, N, K = 70, 8192, 16_384
    W = F.QuantizedMx4.empty(E, N, K)
    W.codes.zero_()
    W.scale.fill_(127)
    last = matrix(N, K, 3)
    one = operand(*last, K)
    W.codes[E - 1], W.scale[E - 1] = one.codes, one.scale
    for T in (3, 200):
        xc = matrix(T, K, 4)
        off = [0] * (E - 1) + [1, T]
        y = torch.full((T, N), 7.0, dtype=BF, device=DEV)
        F.fp8_mx4_grouped_linear_fwd(operand(*xc, K), W, None, offsets_dev(off), y)
        assert not y[0].any()
        xv = X.values(*xc)[1:6]
        r, m = X.linear(xv, X.values(*last))
        check(y[1:6], r, m, "bf16", f"{T}")


class _Guarded:
    """Buffers with 256 bytes of a pattern before and behind."""

    def __init__(self):
        self.kept = []

    def __call__(self, *shape, dtype):
        n = int(np.prod(shape)) * dtype.itemsize
        raw = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device=DEV)
        self.kept.append((raw, n))
        return raw[256:256 + n].view(dtype).view(*shape)

    def check(self):
        for raw, n in self.kept:
            assert (raw[:256] == 0xA5).all() and (raw[256 + n:] == 0xA5).all(), n


@pytest.mark.parametrize("T,E,k", [(1, 5, 2), (31, 96, 6), (33, 257, 3), (700, 64, 8), (9001, 64, 4)])
def test_route_writes_its_outputs_only(T, E, k):
    g = _Guarded()
    z = g(T, E, dtype=torch.float32)
    z.copy_(torch.randn(T, E))
    i32 = torch.int32
    idx, w, off, pos = (g(T, k, dtype=i32), g(T, k, dtype=torch.float32), g(E + 1, dtype=i32),
                        g(T, k, dtype=i32))
    need = F.fp8_route_workspace_bytes(T, E, k)
    ws = g(need, dtype=torch.uint8) if need else None
    F.fp8_route_fwd(z, idx, w, offsets=off, pos=pos, ws=ws)
    dz = g(T, E, dtype=torch.float32)
    F.fp8_route_bwd(z, idx, w, dz)
    F.fp8_route_plan(idx, off, pos, ws=ws)
    for dt, D in ((BF, 33), (torch.float32, 8), (torch.float16, 520)):
        x, xs, y = g(T, D, dtype=dt), g(T * k, D, dtype=dt), g(T, D, dtype=dt)
        x.copy_(torch.randn(T, D))
        F.fp8_route_gather(x, pos, xs)
        F.fp8_route_combine(xs, pos, w, y)
        F.fp8_route_combine_bwd(x, xs, pos, w, g(T * k, D, dtype=dt), g(T, k, dtype=torch.float32))
    torch.cuda.synchronize()
    g.check()


@pytest.mark.parametrize("dt", [BF, torch.float16])
@pytest.mark.parametrize("M,N,K", [(1, 33, 70), (5, 96, 1003), (17, 250, 129), (130, 77, 33),
                                   (300, 520, 544), (1000, 272, 100)])
def test_4_bit_layers_write_their_outputs_only(M, N, K, dt):
    g = _Guarded()
    u8 = torch.uint8

    def empty(*shape):
        *lead, r, c = shape
        return F.QuantizedMx4(g(*lead, r, 16 * -(-c // 32), dtype=u8),
                              g(*lead, -(-c // 128), r, 4, dtype=u8), c)

    E = 3
    wt, x = g(E, N, K, dtype=dt), g(M, K, dtype=dt)
    wt.copy_(torch.randn(E, N, K))
    x.copy_(torch.randn(M, K))
    W, q = empty(E, N, K), empty(M, K)
    F.fp8_mx4_quantize(wt, W.codes, W.scale)
    F.fp8_mx4_dequantize(W, g(E, N, K, dtype=dt))
    off = offsets_dev([0, M // 3, M // 3, M])
    F.fp8_mx4_grouped_linear_fwd(x, W, g(E, N, dtype=dt), off, g(M, N, dtype=dt), q.codes, q.scale)
    one = F.QuantizedMx4(W.codes[0], W.scale[0], K)
    F.fp8_mx4_linear_fwd(x, one, None, g(M, N, dtype=dt), q.codes, q.scale)
    torch.cuda.synchronize()
    g.check()
