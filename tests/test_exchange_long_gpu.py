"""Sums along the longest rows that the exchange takes, of values whose sums
round at every step."""

import pytest
import torch

import scaled_quantize_fp8_amd as F
from tests.gpu_util import DEV
from tests.test_exchange_gpu import DT, HALF

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("D", [1 << 22, (1 << 22) - 5, 100_003])
@pytest.mark.parametrize("sign", ["both", "one"])
def test_gradients_along_long_rows(D, dt, sign):
    """A lane adds D / 64 products (a few more where the last piece overlaps the
    one before) to its sum by fused steps, 64 lanes join in six: a product is
    in at most D / 64 + 8 + 6 roundings of 2^-24."""
    T, k = 3, 2
    g = torch.Generator(device=DEV).manual_seed(D)
    rand = lambda *s: torch.randn(*s, generator=g, device=DEV)
    y, dout = rand(T * k, D).to(DT[dt]), rand(T, D).to(DT[dt])
    if sign == "one":  # sums that grow: every step rounds at their size
        y, dout = y.abs(), dout.abs()
    w = rand(T, k)
    pos = torch.tensor([[5, 0], [2, 4], [1, 3]], dtype=torch.int32, device=DEV)
    dy, dw = torch.empty_like(y), torch.empty(T, k, device=DEV)
    F.fp8_route_combine_bwd(dout, y, pos, w, dy, dw)
    p = dout.double()[:, None] * y.double()[pos.long()]
    r, mag = p.sum(2), p.abs().sum(2)
    assert ((dw.double() - r).abs() <= 2.0 ** -24 * (D / 64 + 16) * mag).all()
    ry = w.double()[:, :, None] * dout.double()[:, None]
    err = (dy.double()[pos.long()] - ry).abs()
    tiny = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25, "fp32": 2.0 ** -150}[dt]
    # w dout in 32 bits, then the type's rounding
    assert (err <= (HALF[dt] * (1 + 2.0 ** -24) + 2.0 ** -24) * ry.abs() + tiny).all()
