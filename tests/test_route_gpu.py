"""Routing to experts on the GPU: choices and places equal to the oracle's,
weights and gradients within the bound that the arithmetic allows."""

import numpy as np
import pytest
import torch

import scaled_quantize_fp8_amd as F
from oracle import route_oracle as R
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25, "fp32": 2.0 ** -126}


def _logits(T, E, dt, seed, kind="normal"):
    rng = np.random.default_rng(seed)
    z = rng.standard_normal((T, E)) * 2
    if kind == "ties":
        z = np.rint(z)
    if kind == "wide":
        z = z * 40
    return torch.from_numpy(z).to(DT[dt])


def _bias(E, seed, kind="normal"):
    rng = np.random.default_rng(seed)
    b = np.float32(rng.standard_normal(E) * 0.1)
    return np.float32(np.rint(b * 10) * 0.125) if kind == "ties" else b


def _route(z, k, bias=None, plan=True, **kw):
    T, E = z.shape
    zd = z.to(DEV)
    idx = torch.full((T, k), 77, dtype=torch.int32, device=DEV)
    w = torch.full((T, k), -7.0, device=DEV)
    off = torch.full((E + 1,), 99, dtype=torch.int32, device=DEV) if plan else None
    pos = torch.full((T, k), 99, dtype=torch.int32, device=DEV) if plan else None
    ws = torch.empty(max(4, F.fp8_route_workspace_bytes(T, E, k)), dtype=torch.uint8, device=DEV)
    b = None if bias is None else torch.from_numpy(bias).to(DEV)
    F.fp8_route_fwd(zd, idx, w, bias=b, offsets=off, pos=pos, ws=ws, **kw)
    torch.cuda.synchronize()
    return idx, w, off, pos


def _check(z, bias, k, idx, w, score=0, groups=1, groups_kept=1, group_top=1, renorm=True,
           scale=1.0):
    zs = z.to(torch.float64).numpy()
    got, wg = idx.cpu().numpy(), w.cpu().to(torch.float64).numpy()
    for t in range(zs.shape[0]):
        want = R.choose(zs[t], bias, score, k, groups, groups_kept, group_top)
        assert got[t].tolist() == want, f"row {t}: {got[t]} for {want}"
        r, rel = R.weights(zs[t], want, score, renorm, scale)
        if bias is not None and np.isnan(bias).any():
            r = np.full(k, np.nan)
        nan = np.isnan(r)
        assert np.array_equal(np.isnan(wg[t]), nan), f"row {t}: NaN weights differ"
        bad = ~(np.abs(wg[t] - r) <= 2.0 ** -24 * rel * np.abs(r) + 2.0 ** -126 * scale) & ~nan
        assert not bad.any(), f"row {t}: {wg[t][bad]} for {r[bad]}"


def _check_places(idx, off, pos, E):
    o, p = R.places(idx.cpu().numpy(), E)
    assert np.array_equal(off.cpu().numpy(), o) and np.array_equal(pos.cpu().numpy(), p)


SIZES = [(1, 1, 1), (1, 64, 4), (3, 8, 2), (33, 17, 5), (130, 96, 6), (70, 256, 8), (9, 200, 16),
         (5, 40, 20), (6, 64, 64), (21, 257, 3), (4, 600, 33), (18, 1024, 8)]


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("T,E,k", SIZES)
def test_choice_weights_places(T, E, k, biased, score, dt):
    z, b = _logits(T, E, dt, T + E), _bias(E, E) if biased else None
    kw = dict(score=score, renorm=bool((T + k) % 2), scale=2.5)
    idx, w, off, pos = _route(z, k, b, **kw)
    _check(z, b, k, idx, w, **kw)
    _check_places(idx, off, pos, E)


@pytest.mark.parametrize("kind", ["normal", "ties", "wide"])
@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("E,groups,kept,k", [(256, 8, 4, 8), (96, 3, 2, 6), (60, 12, 5, 7),
                                             (64, 64, 9, 9), (512, 16, 1, 32), (40, 8, 8, 4),
                                             (1024, 8, 3, 8)])
@pytest.mark.parametrize("top", [1, 2])
def test_groups(E, groups, kept, k, top, biased, score, kind):
    T = 23
    z, b = _logits(T, E, "fp32", E + top, kind), _bias(E, E, kind) if biased else None
    kw = dict(score=score, groups=groups, groups_kept=kept, group_top=top)
    idx, w, _, _ = _route(z, k, b, plan=False, **kw)
    _check(z, b, k, idx, w, **kw)


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("biased", [False, True])
def test_ties_go_to_the_lowest_index(score, biased):
    z, b = _logits(64, 130, "bf16", 5, "ties"), _bias(130, 6, "ties") if biased else None
    idx, w, _, _ = _route(z, 12, b, plan=False, score=score)
    _check(z, b, 12, idx, w, score=score)
    z = torch.zeros(7, 256, dtype=torch.bfloat16)
    idx, _, _, _ = _route(z, 8, None if b is None else np.float32(np.full(256, 0.25)), plan=False,
                          score=score)
    assert (idx.cpu().numpy() == np.arange(8)).all()


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("E", [64, 256, 700])
def test_scores_closer_than_32_bits(score, E):
    """Logits one step of fp32 apart with a common bias: in 32 bits most scores
    would be equal."""
    rng = np.random.default_rng(E)
    base = np.float32(6.0) if score else np.float32(1.0)
    steps = np.stack([rng.permutation(E) for _ in range(40)])
    z = torch.from_numpy(base + np.float32(steps) * np.spacing(base))
    for b in (np.full(E, np.float32(0.3)), np.float32(rng.integers(0, 2, E) * 0.5)):
        idx, w, _, _ = _route(z, 8, b, plan=False, score=score)
        _check(z, b, 8, idx, w, score=score)


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("T", [1, 5, 33, 70])
@pytest.mark.parametrize("E,groups", [(16, 4), (64, 8), (48, 4), (96, 12), (128, 4), (160, 8),
                                      (256, 8), (255, 5), (600, 8)])
def test_groups_closer_than_32_bits(E, groups, T, score):
    """Every third row as above, others ordinary ones: groups, and experts of
    them, that 32 bits do not tell apart; whole, in parts of a lane's experts
    and over lanes."""
    rng = np.random.default_rng(E + T)
    base = np.float32(6.0) if score else np.float32(1.0)
    z = np.float32(2 * rng.standard_normal((T, E)))
    z[::3] = base + np.float32(rng.integers(0, 40, z[::3].shape)) * np.spacing(base)
    z = torch.from_numpy(z)
    for b in (None, np.full(E, np.float32(0.3))):
        for top in (1, 2):
            kw = dict(score=score, groups=groups, groups_kept=groups // 2, group_top=top)
            idx, w, _, _ = _route(z, 4, b, **kw)
            _check(z, b, 4, idx, w, **kw)


@pytest.mark.parametrize("score", [0, 1])
def test_saturated_and_underflowing_scores(score):
    rng = np.random.default_rng(2)
    z = np.concatenate([30 + rng.standard_normal((20, 48)), -150 + 20 * rng.standard_normal((20, 48)),
                        rng.choice([-300.0, 0.0, 300.0], (20, 48)) + rng.standard_normal((20, 48))])
    z = torch.from_numpy(np.float32(z))
    for b in (None, np.float32(rng.choice([0.0, 0.25], 48))):
        for renorm in (True, False):
            idx, w, _, _ = _route(z, 6, b, plan=False, score=score, renorm=renorm)
            _check(z, b, 6, idx, w, score=score, renorm=renorm)


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("E,k,groups", [(24, 4, 1), (24, 4, 3), (300, 18, 1)])
def test_masks_and_values_that_are_not_finite(E, k, groups, dt, score):
    z = _logits(12, E, dt, 3)
    low, inf, nan = torch.finfo(DT[dt]).min, float("inf"), float("nan")
    z[0] = -inf
    z[1, 3:] = -inf
    z[2] = low
    z[3, 1:] = low
    z[4, 5] = nan
    z[5, E - 1] = inf
    z[6, 7], z[6, 9] = inf, inf
    z[7, ::2] = -inf
    z[8] = nan
    z[9, :E - 2] = -inf
    z[10, 2] = torch.finfo(DT[dt]).max
    kw = dict(score=score, groups=groups, groups_kept=max(1, groups - 1))
    for b in (None, _bias(E, 4)):
        if b is not None:
            b[::5] = -np.inf
        idx, w, off, pos = _route(z, k, b, **kw)
        _check(z, b, k, idx, w, **kw)
        _check_places(idx, off, pos, E)
    b = _bias(E, 4)
    b[2] = np.nan
    idx, w, _, _ = _route(z, k, b, plan=False, **kw)
    assert (idx.cpu().numpy() == np.arange(k)).all() and torch.isnan(w).all()


def test_no_tokens():
    z = torch.zeros(0, 8)
    idx, w, off, pos = _route(z, 2)
    assert off.tolist() == [0] * 9
    F.fp8_route_bwd(z.to(DEV), idx, w, torch.empty(0, 8, device=DEV))


def _check_bwd(z, idx, dw, dt, score, renorm, scale):
    dz = torch.full(z.shape, 5.0, dtype=z.dtype, device=DEV)
    F.fp8_route_bwd(z.to(DEV), idx, torch.from_numpy(dw).to(DEV), dz, score=score, renorm=renorm,
                    scale=scale)
    got, zs, ix = dz.cpu().to(torch.float64).numpy(), z.to(torch.float64).numpy(), idx.cpu().numpy()
    for t in range(z.shape[0]):
        r, d = R.gradient(zs[t], ix[t], dw[t], score, renorm, scale)
        tol = d + HALF[dt] * (np.abs(r) + d) + TINY[dt] + 2.0 ** -126
        bad = ~(np.abs(got[t] - r) <= tol)
        assert not bad.any(), f"row {t}: {got[t][bad][:4]} for {r[bad][:4]}"


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,E,k", SIZES)
def test_gradient(T, E, k, renorm, score, dt):
    z = _logits(T, E, dt, T * 3 + E)
    idx, _, _, _ = _route(z, k, plan=False, score=score)
    idx[T // 2, k // 2] = -1  # a slot without an expert
    dw = np.float32(np.random.default_rng(E).standard_normal((T, k)))
    _check_bwd(z, idx, dw, dt, score, renorm, 1.5)


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_of_padding_masks_and_repeats(score, renorm):
    z = _logits(6, 20, "fp32", 1)
    z[0] = -float("inf")
    z[1, 4:] = -float("inf")
    idx = torch.tensor([[-1, -1, -1], [0, 3, -1], [5, 5, 2], [19, 0, 25], [-9, 1, 1], [7, 8, 9]],
                       dtype=torch.int32, device=DEV)
    dw = np.float32(np.random.default_rng(0).standard_normal((6, 3)))
    ok = idx.cpu().clone()
    ok[ok >= 20] = -1
    ok[ok < 0] = -1
    dz = torch.empty(6, 20, device=DEV)
    F.fp8_route_bwd(z.to(DEV), idx, torch.from_numpy(dw).to(DEV), dz, score=score, renorm=renorm)
    again = torch.empty(6, 20, device=DEV)
    F.fp8_route_bwd(z.to(DEV), ok.to(DEV), torch.from_numpy(dw).to(DEV), again, score=score,
                    renorm=renorm)
    assert torch.equal(dz, again) and not dz[0].any()
    _check_bwd(z, ok.to(DEV), dw, "fp32", score, renorm, 1.0)


@pytest.mark.parametrize("T,k,E", [(0, 3, 5), (1, 1, 1), (1, 64, 1024), (683, 3, 7), (2048, 1, 64),
                                   (2049, 1, 1), (5000, 8, 64), (3001, 7, 1000), (262144, 5, 96)])
def test_places_of_any_index(T, k, E):
    rng = np.random.default_rng(T + E)
    idx = torch.from_numpy(rng.integers(-2, E + 2, (T, k)).astype(np.int32)).to(DEV)
    off = torch.full((E + 1,), 9, dtype=torch.int32, device=DEV)
    pos = torch.full((T, k), 9, dtype=torch.int32, device=DEV)
    ws = torch.empty(max(4, F.fp8_route_workspace_bytes(T, E, k)), dtype=torch.uint8, device=DEV)
    F.fp8_route_plan(idx, off, pos, ws)
    flat = idx.cpu().numpy().reshape(-1)
    live = np.nonzero((flat >= 0) & (flat < E))[0]
    order = live[np.argsort(flat[live], kind="stable")]
    want = np.full(flat.shape, -1)
    want[order] = np.arange(len(order))
    assert np.array_equal(pos.cpu().numpy().reshape(-1), want)
    assert np.array_equal(np.diff(off.cpu().numpy()), np.bincount(flat[live], minlength=E)[:E])
    assert off[0] == 0
