"""Logits of both zeros: they tie, whatever the type, the number of experts and
the groups, so the lowest index is chosen."""

import numpy as np
import pytest
import torch

from tests.test_route_gpu import DT, _check, _route

pytestmark = pytest.mark.gpu


def _zeros(T, E, seed):
    """Rows of zeros of both signs with a few values above and below."""
    rng = np.random.default_rng(seed)
    z = np.where(rng.random((T, E)) < 0.5, -0.0, 0.0)
    few = rng.random((T, E)) < 0.1
    z[few] = rng.choice([-1.5, 0.75], few.sum())
    z[0] = -0.0
    z[1] = np.where(np.arange(E) % 2 == 0, -0.0, 0.0)
    return z


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("E,k,groups,kept", [(2, 1, 1, 1), (16, 3, 1, 1), (64, 4, 1, 1), (100, 16, 1, 1),
                                             (128, 8, 1, 1), (256, 8, 1, 1), (257, 8, 1, 1), (64, 20, 1, 1),
                                             (256, 8, 8, 4), (160, 6, 8, 3), (60, 7, 12, 5), (16, 4, 4, 2),
                                             (320, 8, 8, 3)])
@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("T", [9, 50])
def test_zeros_of_both_signs_tie(T, top, E, k, groups, kept, score, dt):
    z = torch.from_numpy(_zeros(T, E, E + k)).to(DT[dt])
    assert torch.signbit(z[0]).all()
    for b in (None, np.float32(np.where(np.arange(E) % 3 == 0, -0.0, 0.0))):
        kw = dict(score=score, groups=groups, groups_kept=kept, group_top=top)
        idx, w, _, _ = _route(z, k, b, **kw)
        _check(z, b, k, idx, w, **kw)
