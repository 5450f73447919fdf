"""Routing of more rows than one launch takes (2^32 threads), and of a few more
than one part of them."""

import numpy as np
import pytest
import torch

import scaled_quantize_fp8_amd as F
from oracle import route_oracle as R
from tests.gpu_util import DEV, f32

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.mark.parametrize("T,E,k,dt", [((1 << 24) + 37, 6, 2, torch.float32), ((1 << 24) + 3, 257, 2, BF),
                                      ((1 << 26) + 9, 257, 2, BF), ((1 << 28) + 21, 2, 1, BF)])
def test_rows_past_one_launch(T, E, k, dt):
    """Rows whose k best experts are known: choice, weights, places and gradient
    of all of them."""
    z = torch.zeros(T, E, dtype=dt, device=DEV)
    rows = torch.arange(T, device=DEV)
    best = (rows * 7919 + rows // 4099) % E
    want = torch.stack([best, (best + 1) % E], 1)[:, :k].to(torch.int32)
    z.scatter_(1, want.long(), torch.tensor([3.0, 2.0], device=DEV)[:k].to(dt).expand(T, k))
    idx, pos = (torch.full((T, k), 77, dtype=torch.int32, device=DEV) for _ in range(2))
    w, off = torch.full((T, k), 9.0, device=DEV), torch.empty(E + 1, dtype=torch.int32, device=DEV)
    ws = torch.empty(F.fp8_route_workspace_bytes(T, E, k), dtype=torch.uint8, device=DEV)
    F.fp8_route_fwd(z, idx, w, renorm=False, scale=2.0, offsets=off, pos=pos, ws=ws)
    assert torch.equal(idx, want)
    zr = z[0].cpu().to(torch.float64).numpy()
    wr, rel = R.weights(zr, want[0].tolist(), R.SOFTMAX, False, 2.0)
    tol = torch.from_numpy(2.0 ** -24 * rel * wr).to(DEV)
    assert ((w[:5].double() - torch.from_numpy(wr).to(DEV)).abs() <= tol).all()
    # rows of the same values at other experts: the same sums in another order
    assert ((w - w[0]).abs() <= 2 * tol.float()).all()
    flat = want.view(-1)
    count = torch.bincount(flat, minlength=E)
    assert int(off[0]) == 0 and torch.equal(off[1:].long(), count.cumsum(0))
    for e in sorted({0, E // 2, E - 1}):
        mine = pos.view(-1)[flat == e]
        assert torch.equal(mine, torch.arange(len(mine), dtype=torch.int32, device=DEV) + off[e])
    del pos, flat, w
    dz = torch.full_like(z, 5.0)
    dw = torch.tensor([1.0, -0.5], device=DEV)[:k].repeat(T, 1)
    F.fp8_route_bwd(z, idx, dw, dz, renorm=False, scale=2.0)
    half = 2.0 ** -8 if dt is BF else 2.0 ** -24
    for t in (0, 1, (1 << 24) - 1, 1 << 24, T - 2, T - 1):
        r, d = R.gradient(f32(z[t]).astype(np.float64), want[t].tolist(), np.array([1.0, -0.5])[:k],
                          R.SOFTMAX, False, 2.0)
        assert (np.abs(f32(dz[t]) - r) <= d + half * (np.abs(r) + d)).all(), t
    # the other rows: what row 0 has at its experts and beside them
    got = dz.gather(1, want.long())
    near = torch.tensor([2.0 ** -6], device=DEV).to(dt)
    assert ((got - got[0]).abs() <= near * got[0].abs()).all()
    if E > k:
        dz.scatter_(1, want.long(), dz[0, (int(want[0, -1]) + 1) % E].item())
        rest = dz[0, (int(want[0, -1]) + 1) % E]
        assert (dz.amax(1) - dz.amin(1) <= near * rest.abs()).all()
        assert ((dz[:, 0] - rest).abs() <= near * rest.abs()).all()
