"""A mixture of experts as a model uses it: routing, the exchange of rows and
the grouped layers together, trained in FP8 and served in 4-bit floating point
and 8-bit integers; gradients against the formula's and against differences;
capture, streams, threads."""

import math
import threading

import numpy as np
import pytest
import torch

import scaled_quantize_fp8_amd as F
from oracle import mx4_oracle as X
from oracle import route_oracle as R
from scaled_quantize_fp8_amd import e2e as E
from scaled_quantize_fp8_amd.autograd import Fp8GroupedLinear, Fp8Linear
from scaled_quantize_fp8_amd.int8 import Int8GroupedLinear, Int8Linear
from scaled_quantize_fp8_amd.mixture import Mixture, Router, combine, dispatch, route
from scaled_quantize_fp8_amd.mx4 import Mx4GroupedLinear, Mx4Linear
from tests.gpu_util import DEV, f32
from tests.mx4_util import check
from tests.rows_util import bf16

pytestmark = pytest.mark.gpu

SETTINGS = [dict(), dict(renorm=False), dict(score="sigmoid", scale=2.5),
            dict(score="sigmoid", renorm=False),
            dict(score="sigmoid", groups=4, groups_kept=2, group_top=2)]


def _plain_weights(z, idx, score="softmax", renorm=True, scale=1.0, **_):
    """Weights [T, k] of a given choice in 64 bits, with their gradient."""
    live = idx >= 0
    at = idx.clamp(min=0).long()
    p = z.double().softmax(1) if score == "softmax" else z.double().sigmoid()
    w = torch.where(live, p.gather(1, at), torch.zeros((), dtype=torch.float64, device=z.device))
    if renorm:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    return w * scale


def _apart(T, n, step, seed):
    """Logits whose values in a row are at least `step` apart."""
    rng = np.random.default_rng(seed)
    return np.stack([(rng.permutation(n) - n / 2) * step for _ in range(T)])


@pytest.mark.parametrize("how", SETTINGS)
def test_route_gradient_against_differences(how):
    """f = sum g w over one row, |g| <= 1, k = 3.  The kernel's f is off by
    2^-20 (16 roundings of 2^-24 on weights that sum to at most `scale`, taken
    with it), so a difference over 2h = 2^-6 by 2^-13.  It differs from the
    slope by h^2 / 6 times the third derivative, for logits in [-2, 2] at most
    7 `scale` (sigmoids of at least 0.12, a sum of at least 0.36 as divisor):
    2^-13.8.  The sum of both is below 2^-12."""
    T, n, k = 3, 16, 3
    scale = how.get("scale", 1.0)
    z = _apart(T, n, 0.25, 1)
    g = np.random.default_rng(2).uniform(-1, 1, (T, k))
    gd = torch.from_numpy(g).float().to(DEV)

    def f(v):
        w, idx, _, _ = route(torch.from_numpy(v).float().to(DEV), k, **how)
        return (w.double().cpu().numpy() * gd.double().cpu().numpy()).sum(1), idx

    zt = torch.from_numpy(z).float().to(DEV).requires_grad_(True)
    w, idx, _, _ = route(zt, k, **how)
    w.backward(gd)
    h = 2.0 ** -7
    for e in range(n):
        hi, lo = z.copy(), z.copy()
        hi[:, e] += h
        lo[:, e] -= h
        (a, ia), (b, ib) = f(hi), f(lo)
        assert torch.equal(ia, idx) and torch.equal(ib, idx)
        d = (a - b) / (2 * h)
        got = zt.grad[:, e].double().cpu().numpy()
        assert (np.abs(got - d) <= 2.0 ** -12 * scale).all(), (e, got, d)


@pytest.mark.parametrize("how", SETTINGS)
@pytest.mark.parametrize("T,n,k,D", [(1, 16, 1, 8), (37, 16, 4, 72), (300, 64, 6, 40)])
def test_gradients_through_the_exchange(T, n, k, D, how):
    """route, dispatch, an expert's function, combine: outputs and gradients of
    tokens and logits against the same in 64 bits; some tokens are padding.
    fp32 throughout; the sums here are of at most k + D + n terms, each off by
    a few units: (k + D + n + 64) 2^-24 of the sum of magnitudes."""
    rng = np.random.default_rng(T + n)
    z = _apart(T, n, 1 / 16, 3)
    z[T // 2:T // 2 + T // 8] = -np.inf
    z = torch.from_numpy(z).float().to(DEV).requires_grad_(True)
    x = torch.from_numpy(rng.standard_normal((T, D))).float().to(DEV).requires_grad_(True)
    g = torch.from_numpy(rng.standard_normal((T, D))).float().to(DEV)
    a = torch.from_numpy(rng.standard_normal((n, D))).float().to(DEV)

    w, idx, pos, off = route(z, k, **how)
    xs = dispatch(x, pos)
    of_row = torch.zeros(T * k, dtype=torch.long, device=DEV)
    live = idx >= 0
    of_row[pos[live].long()] = idx[live].long()
    o = off.tolist()
    for e in range(n):  # rows are sorted by expert
        assert (of_row[o[e]:o[e + 1]] == e).all()
    assert not xs[o[-1]:].any() and o[-1] == int(live.sum())
    y = combine(xs * a[of_row], pos, w)
    y.backward(g)

    zp, xp = z.detach().double().requires_grad_(True), x.detach().double().requires_grad_(True)
    with torch.no_grad():
        zp[zp == -math.inf] = -1e300  # the same scores, without NaN in the plain form
    wp = _plain_weights(zp, idx, **how)
    ae = a.double()[idx.clamp(min=0).long()] * live[..., None]
    yp = (wp[..., None] * ae * xp[:, None]).sum(1)
    yp.backward(g.double())
    rel = (k + D + n + 64) * 2.0 ** -24
    scale = how.get("scale", 1.0)
    with torch.no_grad():
        assert ((y - yp).abs() <= rel * (wp[..., None] * (ae * xp[:, None]).abs()).sum(1)).all()
        mag = (wp[..., None] * (ae * g[:, None]).abs()).sum(1)
        assert ((x.grad - xp.grad).abs() <= rel * mag).all()
        # a logit's gradient: weights (below scale) times sums over D, twice
        size = scale * (ae * xp[:, None] * g[:, None]).abs().sum((1, 2))
        assert ((z.grad - zp.grad).abs() <= 2 * rel * size[:, None]).all()
    assert not x.grad[~live.any(1)].any() and not z.grad[~live.any(1)].any()


def test_strided_inputs_and_broadcast_gradients():
    """Transposed logits, a slice of the tokens, expanded gradients."""
    T, n, k, D = 20, 24, 3, 40
    z = torch.from_numpy(_apart(T, n, 1 / 16, 5)).float().to(DEV)
    x = torch.randn(T, 2 * D, device=DEV)
    ref = None
    for zz, xx in ((z, x[:, :D].clone()), (z.T.contiguous().T, x[:, :D])):
        zz, xx = zz.detach().requires_grad_(True), xx.detach().requires_grad_(True)
        w, _, pos, _ = route(zz, k)
        y = combine(dispatch(xx, pos), pos, w)
        y.sum().backward()  # an expanded gradient
        got = y.detach(), zz.grad, xx.grad
        assert ref is None or all(torch.equal(a, b) for a, b in zip(got, ref))
        ref = got
    # frozen tokens: the weights' gradient alone, and the reverse
    for freeze_x in (True, False):
        zz, xx = z.clone().requires_grad_(not freeze_x), x[:, :D].clone().requires_grad_(freeze_x)
        w, _, pos, _ = route(zz, k)
        combine(dispatch(xx, pos), pos, w).sum().backward()
        assert torch.equal(xx.grad, ref[2]) if freeze_x else torch.equal(zz.grad, ref[1])


def test_no_tokens():
    x = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    w, idx, pos, off = route(torch.empty(0, 8, device=DEV), 2)
    assert w.shape == (0, 2) and not off.any()
    assert combine(dispatch(x, pos), pos, w).shape == (0, 64)


def _mixture(d=96, ffn=160, experts=6, k=2, seed=70, **how):
    m = Mixture(d, ffn, experts, k, device=DEV, **how)
    with torch.no_grad():
        for s, p in enumerate(m.parameters()):
            p.copy_(bf16(p.shape, 0.05, seed + s))
        m.router.weight.mul_(4)
    return m


def _cos(a, b):
    a, b = a.detach().double().flatten(), b.detach().double().flatten()
    return float(a @ b / (a.norm() * b.norm()))


def _plain_mixture(m, x):
    """The mixture in 64 bits with m's choice of experts: output, parameters."""
    p = {n: v.detach().double().requires_grad_(True) for n, v in m.named_parameters()}
    with torch.no_grad():
        _, idx, _, _ = m.router(x.detach().to(torch.bfloat16))
    w = _plain_weights(x @ p["router.weight"].T, idx)
    at = idx.clamp(min=0).long()
    every = torch.einsum("td,ehd->teh", x, p["up.weight"]) + p["up.bias"]
    every = torch.nn.functional.gelu(every)
    every = torch.einsum("teh,edh->ted", every, p["down.weight"]) + p["down.bias"]
    mine = every.gather(1, at[..., None].expand(-1, -1, x.shape[1]))
    return (w[..., None] * mine).sum(1), p


def test_mixture_trains_in_fp8():
    """Two steps: the output and every gradient point where the 64-bit
    mixture's do (the cosines asked of the dense and the grouped layers); an
    expert that the router bars gets zero gradients."""
    m = _mixture(bias=True)
    m.router.bias[4] = -math.inf
    for step in range(2):
        x = bf16((5, 40, 96), 1.0 + step, 90 + step).to(DEV).requires_grad_(True)
        g = bf16((5, 40, 96), 1e-3, 95 + step).to(DEV)
        m.zero_grad(set_to_none=True)
        y = m(x)
        y.backward(g)
        xp = x.detach().double().view(200, 96).requires_grad_(True)
        yp, p = _plain_mixture(m, xp)
        yp.backward(g.double().view(200, 96))
        assert y.shape == x.shape and _cos(y, yp) > 0.99 and _cos(x.grad, xp.grad) > 0.98
        for name, v in m.named_parameters():
            assert _cos(v.grad, p[name].grad) > 0.98, name
            if name != "router.weight":
                assert not v.grad[4].any()


def test_trained_mixture_served_in_4_bits_stage_by_stage():
    """Every stage against the oracle on that stage's own input; the module's
    output is the stages' run."""
    d, ffn, n, k, T = 96, 160, 6, 2, 45
    mix = _mixture(d, ffn, n, k, bias=True)
    mix(bf16((64, d), 1.0, 1).to(DEV)).sum().backward()
    mix.router.bias[1] = -math.inf
    m = mix.served(Mx4GroupedLinear)
    x = bf16((T, d), 1.0, 2).to(DEV)
    with torch.no_grad():
        z = torch.nn.functional.linear(x, m.router.weight)
        w, idx, pos, off = m.router(x)
        xs = dispatch(x, pos)
        h = m.up(xs, off)
        act = torch.nn.functional.gelu(h)
        ys = m.down(act, off)
        y = m(x)
    zs, bias = f32(z).astype(np.float64), m.router.bias.cpu().numpy()
    want = [R.choose(zs[t], bias, 0, k) for t in range(T)]
    assert idx.cpu().tolist() == want
    o, p = R.places(np.array(want), n)
    assert off.cpu().tolist() == o.tolist() and np.array_equal(pos.cpu().numpy(), p)
    assert o[2] == o[1]  # the barred expert
    assert np.array_equal(f32(xs), R.gather(f32(x), p, np.zeros((T * k, d), np.float32)))
    for got, rows, lin in ((h, xs, mix.up), (ys, act, mix.down)):
        rv = X.values(*X.quantize(f32(rows)))
        for e in range(n):
            i, j = o[e], o[e + 1]
            if j > i:
                we = X.values(*X.quantize(f32(lin.weight.detach()[e])))
                r, mag = X.linear(rv[i:j], we, f32(lin.bias.detach())[e])
                check(got[i:j], r, mag, "bf16", f"expert {e}")
    r, mag = R.combine(f32(ys).astype(np.float64), p, w.cpu().numpy())
    tol = 2.0 ** -24 * k * mag
    assert (np.abs(f32(y) - r) <= tol + 2.0 ** -8 * (np.abs(r) + tol) + 2.0 ** -134).all()


def test_weights_that_4_bits_hold_are_taken_over_exactly():
    """A dense layer of values that the format holds: the codes stand for the
    weight itself; outputs against the oracle; no gradient."""
    rng = np.random.default_rng(4)
    v = rng.choice([0, .5, 1, 1.5, 2, 3, 4, 6, -1, -3, -6], (72, 100))
    v[:, ::32] = 6
    lin = Fp8Linear(100, 72, device=DEV)
    with torch.no_grad():
        lin.weight.copy_(torch.from_numpy(v))
    m = Mx4Linear.from_linear(lin, torch.float16)
    assert torch.equal(m.dequantize(), lin.weight.detach())
    x = bf16((2, 5, 100), 1.0, 6).to(DEV)
    y = m(x)
    assert y.shape == (2, 5, 72) and y.dtype == torch.float16
    r, mag = X.linear(X.values(*X.quantize(f32(x).reshape(10, 100)))[:, :100], v,
                      f32(lin.bias.detach()))
    check(y.view(10, 72), r, mag, "fp16")
    assert torch.equal(m(x[:0]), y[:0])
    with pytest.raises(RuntimeError, match="no gradient"):
        m(x.clone().requires_grad_(True))
    with torch.no_grad():
        assert torch.equal(m(x.clone().requires_grad_(True)), y)
    again = Mx4Linear.from_linear(Fp8Linear(100, 72, device=DEV), torch.float16)
    again.load_state_dict(m.state_dict())
    assert torch.equal(again(x), y)


def test_router_settings_and_refusals():
    r = Router(32, 16, 4, bias=True, device=DEV, score="sigmoid", groups=4, groups_kept=2)
    w, idx, _, _ = r(bf16((9, 32), 1.0, 1).to(DEV))
    assert ((idx // 4).sort(1).values.diff(dim=1) != 0).sum(1).le(1).all()  # at most two groups
    assert "bias" in r.state_dict() and not r.bias.requires_grad
    z = torch.zeros(4, 8, device=DEV)
    with pytest.raises(ValueError, match="score"):
        route(z, 2, score="tanh")
    with pytest.raises(F.Fp8Error):
        route(z, 9)
    with pytest.raises(F.Fp8Error):
        route(z, 2, groups=3)
    with pytest.raises(ValueError):
        route(z, 2, bias=torch.zeros(7, device=DEV))
    with pytest.raises((TypeError, ValueError)):
        route(z.double(), 2)
    _, _, pos, _ = route(z, 2)
    with pytest.raises(ValueError):
        combine(torch.zeros(8, 16, device=DEV), pos, torch.ones(4, 3, device=DEV))


def _small(lin, experts):
    return E.Transformer(lin, layers=2, d=128, heads=4, ffn=256, vocab=200, device=DEV,
                         experts=experts, k=2)


@pytest.mark.parametrize("kinds", [(Mx4Linear, Mx4GroupedLinear), (Int8Linear, Int8GroupedLinear)])
@pytest.mark.parametrize("experts", [0, 5])
def test_transformer_trains_and_is_served(experts, kinds):
    """Runs, every parameter has a finite gradient that is not zero, and the
    quantized model runs without one."""
    m = _small(E.fp8_linear, experts)
    tok, tgt = E.synthetic_batch(2, 64, 200, DEV, seed=9)
    with E.attention_backends():
        for _ in range(2):
            m.zero_grad(set_to_none=True)
            m.loss(tok, tgt).backward()
        for name, p in m.named_parameters():
            assert p.grad is not None and p.grad.isfinite().all() and p.grad.any(), name
        s = E.served(m, *kinds)
        with torch.no_grad():
            for t in (tok, tok[:1, :1]):
                z = s.logits(t)
                assert z.shape == (*t.shape, 200) and z.isfinite().all()
    assert not any(p.requires_grad for p in s.parameters())


def test_training_step_replays_like_eager_steps():
    dims = dict(layers=1, d=128, heads=4, ffn=256, vocab=200, experts=5, k=2)
    eager, _ = E.train(E.fp8_linear, 4, DEV, graph=False, dims=dims, batch=(2, 64))
    replay, _ = E.train(E.fp8_linear, 4, DEV, graph=True, dims=dims, batch=(2, 64))
    assert len(replay) == 4 and eager == replay


def test_captured_backward_beside_a_living_eager_graph():
    """Forward and backward of the mixture captured while an eager graph of the
    same parameters is alive; between the replays the tokens and with them the
    choice of experts change, and eager work runs."""
    m = _mixture()
    xs = [bf16((70, 96), 1.0, 20 + i).to(DEV) for i in range(3)]
    x, g = xs[0].clone(), bf16((70, 96), 1e-3, 2).to(DEV)
    ps = list(m.parameters())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(3):
            m.zero_grad(set_to_none=True)
            m(x).backward(g)
    torch.cuda.current_stream().wait_stream(s)
    m.zero_grad(set_to_none=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = m(x)
        grads = torch.autograd.grad(y, ps, g)
    alive = m(x.clone())

    def rings():
        return [r for lin in (m.up, m.down) for r in (lin.ring_x, lin.ring_w, lin.ring_g)]

    for i in range(4):
        x.copy_(xs[i % 3])
        saved = [r.buf.clone() for r in rings()]
        graph.replay()
        torch.cuda.synchronize()
        for r, v in zip(rings(), saved):  # the same scales again
            r.buf.copy_(v)
        y2 = m(x)
        want = torch.autograd.grad(y2, ps, g)
        torch.cuda.synchronize()
        assert torch.equal(y, y2), i
        assert all(torch.equal(a, b) for a, b in zip(grads, want)), i
    alive.backward(g)
    assert all(p.grad is not None for p in ps)


def test_capture_beside_an_eager_graph_of_another_stream_is_refused():
    """A graph of the same leaves built before the capture, on another stream:
    each entry refuses before anything of a backward is captured; once that
    graph is gone the same capture works."""
    m = _mixture()
    x, g = bf16((70, 96), 1.0, 1).to(DEV), bf16((70, 96), 1e-3, 2).to(DEV)
    z = torch.randn(6, 8, device=DEV).requires_grad_(True)
    v = torch.randn(6, 16, device=DEV).requires_grad_(True)
    ys = torch.randn(12, 16, device=DEV).requires_grad_(True)
    w, _, pos, _ = (t.detach() for t in route(z.detach(), 2))
    calls = [lambda: m(x), lambda: m.router(x)[0], lambda: route(z, 2)[0],
             lambda: dispatch(v, pos), lambda: combine(ys, pos, w)]
    for call in calls:
        alive = call()
        torch.cuda.synchronize()
        with pytest.raises(RuntimeError, match="living eager graph"):
            with torch.cuda.graph(torch.cuda.CUDAGraph()):
                call()
        torch.cuda.synchronize()
        del alive
    ps = list(m.parameters())
    want = torch.autograd.grad(m(x), ps, g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        grads = torch.autograd.grad(m(x), ps, g)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(grads, want))


def _serve_calls(T, n, k, d, ffn, seed):
    """A served block's buffers, and a function that enqueues its calls on a stream."""
    mix = _mixture(d, ffn, n, k, seed=seed).served(Mx4GroupedLinear)
    x = bf16((T, d), 1.0, seed).to(DEV)
    z = torch.nn.functional.linear(x, mix.router.weight.detach())
    e = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device=DEV)
    idx, pos, off = e(T, k, dt=torch.int32), e(T, k, dt=torch.int32), e(n + 1, dt=torch.int32)
    w, xs, h, ys, y = e(T, k, dt=torch.float32), e(T * k, d), e(T * k, ffn), e(T * k, d), e(T, d)
    ws = e(max(4, F.fp8_route_workspace_bytes(T, n, k)), dt=torch.uint8)
    qx, qh = F.QuantizedMx4.empty(T * k, d), F.QuantizedMx4.empty(T * k, ffn)
    up, down = mix.up._weight(), mix.down._weight()

    def run(stream=None):
        F.fp8_route_fwd(z, idx, w, offsets=off, pos=pos, ws=ws, stream=stream)
        F.fp8_route_gather(x, pos, xs, stream=stream)
        F.fp8_mx4_grouped_linear_fwd(xs, up, mix.up.bias, off, h, qx.codes, qx.scale, stream=stream)
        F.fp8_mx4_grouped_linear_fwd(h, down, mix.down.bias, off, ys, qh.codes, qh.scale,
                                     stream=stream)
        F.fp8_route_combine(ys, pos, w, y, stream=stream)

    return x, z, y, run


SERVED = [(1, 16, 4, 128, 256), (24, 16, 4, 128, 512), (130, 8, 2, 96, 160), (700, 8, 2, 256, 512)]


@pytest.mark.parametrize("T,n,k,d,ffn", SERVED)
def test_served_run_replays_like_eager_ones(T, n, k, d, ffn):
    x, z, y, run = _serve_calls(T, n, k, d, ffn, 5)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for i in range(4):
        x.copy_(bf16((T, d), 1.0, 30 + i))
        z.copy_(bf16((T, n), 1.0, 40 + i))
        y.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        y.fill_(9.0)
        run()
        torch.cuda.synchronize()
        assert torch.equal(got, y), i


def test_served_runs_on_several_streams_and_threads():
    """Four host threads, each on its own stream: what each gives alone."""
    sets = [_serve_calls(*s, 60 + i) for i, s in enumerate(SERVED)]
    want = []
    for _, _, y, run in sets:
        run()
        want.append(y.clone())
        y.zero_()
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    errors = []

    def work(i):
        try:
            torch.cuda.set_device(0)
            for _ in range(5):
                sets[i][3](streams[i])
            streams[i].synchronize()
        except Exception as exc:
            errors.append((SERVED[i], repr(exc)))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(sets))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=100)
    assert not errors, errors
    for (_, _, y, _), v in zip(sets, want):
        assert torch.equal(y, v)


def test_two_captured_graphs_have_their_own_workspaces():
    """Two graphs of more slots than one launch places, replayed on two
    streams at once: each has the workspace its call was given."""
    T, n, k = 9000, 64, 8
    sets = []
    for i in range(2):
        z = bf16((T, n), 1.0, i).to(DEV)
        idx, pos = (torch.empty(T, k, dtype=torch.int32, device=DEV) for _ in range(2))
        w, off = torch.empty(T, k, device=DEV), torch.empty(n + 1, dtype=torch.int32, device=DEV)
        need = F.fp8_route_workspace_bytes(T, n, k)
        assert need > 0
        ws = torch.empty(need, dtype=torch.uint8, device=DEV)
        call = lambda z=z, idx=idx, w=w, off=off, pos=pos, ws=ws: F.fp8_route_fwd(
            z, idx, w, offsets=off, pos=pos, ws=ws)
        call()
        want = off.clone(), pos.clone()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        sets.append((graph, off, pos, want, call))  # call holds the buffers
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        for _, off, pos, *_ in sets:
            off.fill_(-5)
            pos.fill_(-5)
        torch.cuda.synchronize()
        for s, (graph, *_) in zip(streams, sets):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for _, off, pos, (o, p), _ in sets:
            assert torch.equal(off, o) and torch.equal(pos, p)
