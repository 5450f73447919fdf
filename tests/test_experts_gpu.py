"""The experts' layers as a model uses them: routing, the FP8 grouped modules
forward and backward, then the trained weights served in 8-bit integers."""

import numpy as np
import pytest
import torch

import scaled_quantize_fp8_amd as F
from oracle import fp8_oracle as O
from oracle import rows_oracle as R
from scaled_quantize_fp8_amd.autograd import Fp8GroupedLinear, Fp8Linear
from scaled_quantize_fp8_amd.int8 import Int8GroupedLinear, Int8Linear
from tests.gpu_util import DEV, bf16_bits, check_gemm, f32
from tests.rows_util import bf16, check_groups, check_i8, offsets_dev

pytestmark = pytest.mark.gpu


def route(scores, k):
    """Token rows sorted by expert: (token of each row, gate of each row,
    offsets).  scores [tokens, E]."""
    gate, expert = scores.softmax(-1).topk(k)
    expert, order = expert.reshape(-1).sort(stable=True)
    counts = torch.zeros(scores.shape[1], dtype=torch.int64, device=scores.device)
    counts.scatter_add_(0, expert, torch.ones_like(expert))
    off = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    return order // k, gate.reshape(-1)[order], off


def mixture(x, scores, up, down, k=2):
    token, gate, off = route(scores, k)
    h = torch.nn.functional.gelu(up(x[token], off))
    out = down(h, off).float() * gate[:, None]
    return torch.zeros(x.shape, dtype=torch.float32, device=x.device).index_add(0, token, out)


class _Plain(torch.nn.Module):
    """y[t] = x[t] W[e]^T + b[e] in 64 bits."""

    def __init__(self, like):
        super().__init__()
        self.w = torch.nn.Parameter(like.weight.detach().double())
        self.b = torch.nn.Parameter(like.bias.detach().double())

    def forward(self, x, off):
        o = off.tolist()
        return torch.cat([x[o[e]:o[e + 1]].double() @ self.w[e].T + self.b[e]
                          for e in range(len(o) - 1)])


def _cos(a, b):
    a, b = a.double().flatten(), b.double().flatten()
    return float(a @ b / (a.norm() * b.norm()))


def _layers(E=6, D=96, H=160):
    up, down = (Fp8GroupedLinear(E, i, o, device=DEV) for i, o in ((D, H), (H, D)))
    with torch.no_grad():
        for s, p in enumerate([*up.parameters(), *down.parameters()]):
            p.copy_(bf16(p.shape, 0.05, 70 + s))
    return up, down


def test_mixture_trains_in_fp8():
    """Two steps of a routed up / down block: output and every gradient point
    where the 64-bit block's do (cosine above 0.98, as for the dense layers);
    an expert that no token chose gets zero gradients."""
    up, down = _layers()
    T, E, D = 200, 6, 96
    pu, pd = _Plain(up), _Plain(down)
    for step in range(2):
        scores = bf16((T, E), 1.0, 80 + step).float().to(DEV)
        scores[:, 4] = -1e30  # nobody chooses expert 4
        x = bf16((T, D), 1.0 + step, 90 + step).to(DEV).requires_grad_(True)
        xp = x.detach().double().requires_grad_(True)
        g = bf16((T, D), 1e-3, 95 + step).to(DEV)
        for m in (up, down, pu, pd):
            m.zero_grad(set_to_none=True)
        y, yp = mixture(x, scores, up, down), mixture(xp, scores, pu, pd)
        y.backward(g.float())
        yp.backward(g.float())
        assert _cos(y, yp) > 0.99
        assert _cos(x.grad, xp.grad) > 0.98
        for m, p in ((up, pu), (down, pd)):
            assert _cos(m.weight.grad, p.w.grad) > 0.98
            assert _cos(m.bias.grad, p.b.grad) > 0.98
            assert not m.weight.grad[4].any() and not m.bias.grad[4].any()


def test_module_matches_the_oracle():
    """y, dX, dW, db of one step of Fp8GroupedLinear, rows behind the last
    group included (zeros in y and dX)."""
    off, T, E, K, N = [0, 30, 30, 97], 110, 3, 80, 112
    m = Fp8GroupedLinear(E, K, N, device=DEV)
    X, W, b, G = (bf16(s, v, 60 + i) for i, (s, v) in enumerate(
        (((T, K), 1.0), ((E, N, K), 0.02), ((E, N), 0.1), ((T, N), 1e-3))))
    with torch.no_grad():
        m.weight.copy_(W)
        m.bias.copy_(b)
    x = X.to(DEV).requires_grad_(True)
    y = m(x, offsets_dev(off))
    y.backward(G.to(DEV))
    x8, sx, _ = O.quantize_step(f32(X)[:97], O.E4M3, O.ScaleRing(16))
    w8, sw, _ = O.quantize_step(f32(W), O.E4M3, O.ScaleRing(16))
    g8, sg, _ = O.quantize_step(f32(G)[:97], O.E5M2, O.ScaleRing(16))
    check_groups(y, R.grouped_fwd(x8, w8, O.E4M3, sx, [sw], off, f32(b).astype(float)), off, "y")
    check_groups(x.grad, R.grouped_dx(g8, O.E5M2, w8, O.E4M3, sg, [sw], off), off, "dx")
    assert not y[97:].any() and not x.grad[97:].any()
    dbs = R.grouped_db(f32(G)[:97].astype(np.float64), off)
    for e, ref in enumerate(R.grouped_dw(g8, O.E5M2, x8, O.E4M3, sg, sx, off)):
        if ref is None:
            assert not m.weight.grad[e].any() and not m.bias.grad[e].any()
        else:
            check_gemm(bf16_bits(m.weight.grad[e]), ref, "dw")
            check_gemm(bf16_bits(m.bias.grad[e]), dbs[e], "db")


def test_gradients_against_differences():
    """Values that FP8 holds exactly under their own scale (W in {-7, 0, 7}, X
    integers with a 7, G in {-1.75, 0, 1.75}), outputs that bf16 holds exactly:
    central differences of sum(G y) equal dX, dW and db to bf16's half step."""
    rng = np.random.default_rng(11)
    off, E, K, N, T = [0, 3, 3, 5], 3, 8, 4, 5
    X = rng.integers(-2, 3, (T, K)).astype(np.float64)
    X[0, 0] = 7
    W = rng.integers(-1, 2, (E, N, K)) * 7.0
    W[0, 0, 0] = W[2, 0, 0] = 7
    G = rng.integers(-1, 2, (T, N)) * 1.75
    G[0, 0] = 1.75
    m = Fp8GroupedLinear(E, K, N, device=DEV)
    to = lambda a: torch.from_numpy(a).to(torch.bfloat16).to(DEV)

    def f(x, w, b):
        with torch.no_grad():
            m.weight.copy_(to(w))
            m.bias.copy_(to(b))
            m.ring_x = None
            y = m(to(x), offsets_dev(off)).double().cpu().numpy()
        return float((y * G).sum())

    b0 = np.zeros((E, N))
    x = to(X).requires_grad_(True)
    with torch.no_grad():
        m.weight.copy_(to(W))
        m.bias.copy_(to(b0))
    m(x, offsets_dev(off)).backward(to(G))
    got = [g.double().cpu().numpy() for g in (x.grad, m.weight.grad, m.bias.grad)]
    spots = [(0, (1, 3)), (0, (4, 7)), (1, (0, 1, 2)), (1, (2, 3, 5)), (1, (1, 0, 0)),
             (2, (0, 2)), (2, (2, 1)), (2, (1, 1))]
    for which, at in spots:
        hi = [X.copy(), W.copy(), b0.copy()]
        lo = [X.copy(), W.copy(), b0.copy()]
        if which == 1:  # stay on values that the weights' scale holds
            hi[1][at], lo[1][at] = 7.0, -7.0
        else:
            hi[which][at] += 1.0
            lo[which][at] -= 1.0
        d = (f(*hi) - f(*lo)) / (hi[which][at] - lo[which][at])
        assert abs(got[which][at] - d) <= abs(d) * 2.0 ** -8, (which, at, got[which][at], d)


def test_trained_experts_are_served_in_8_bit_integers():
    """The FP8 block's weights through the integer layers: codes as the oracle
    quantizes them, outputs within the integer layer's bound, and the block's
    output close to the 64-bit block's."""
    up, down = _layers()
    T, E, D = 64, 6, 96
    pu, pd = _Plain(up), _Plain(down)
    iu, idn = Int8GroupedLinear.from_grouped(up), Int8GroupedLinear.from_grouped(down)
    oq, os = R.i8_quantize_rows(f32(up.weight.detach()).reshape(-1, D))
    assert np.array_equal(iu.codes.cpu().numpy().reshape(-1, D), oq)
    assert np.array_equal(iu.scale.cpu().numpy().reshape(-1), os)
    x = bf16((T, D), 1.0, 3).to(DEV)
    off = [0, 10, 10, 25, 30, 31, 60]
    y = iu(x, offsets_dev(off))
    xq, xs = R.i8_quantize_rows(f32(x))
    w, sw, b = iu.codes.cpu().numpy(), iu.scale.cpu().numpy(), f32(up.bias.detach())
    for e, i, j in R.spans(off):
        if i < j:
            r, p = R.i8_linear(xq[i:j], xs[i:j], w[e], sw[e], b[e])
            check_i8(y[i:j], r, p, "bf16", f"expert {e}")
    assert not y[60:].any()
    scores = bf16((T, E), 1.0, 4).float().to(DEV)
    with torch.no_grad():
        assert _cos(mixture(x, scores, iu, idn), mixture(x, scores, pu, pd)) > 0.999


def test_dense_layer_is_served_in_8_bit_integers():
    lin = Fp8Linear(128, 72, device=DEV)
    m = Int8Linear.from_linear(lin, torch.float16)
    x = bf16((2, 5, 128), 1.0, 6).to(DEV)
    with torch.no_grad():
        y = m(x)
    assert y.shape == (2, 5, 72) and y.dtype == torch.float16
    xq, xs = R.i8_quantize_rows(f32(x).reshape(10, 128))
    r, p = R.i8_linear(xq, xs, m.codes.cpu().numpy(), m.scale.cpu().numpy(),
                       f32(lin.bias.detach()))
    check_i8(y.view(10, 72), r, p, "fp16")


def test_captured_backward_beside_a_living_eager_graph():
    """A forward and backward captured while an eager autograd graph of the
    same parameters is alive; replays give the eager gradients."""
    off, T, E, K, N = [0, 30, 30, 64], 64, 3, 80, 112
    m = Fp8GroupedLinear(E, K, N, device=DEV)
    x = bf16((T, K), 1.0, 1).to(DEV)
    g = bf16((T, N), 1e-3, 2).to(DEV)
    o = offsets_dev(off)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(3):
            m.zero_grad(set_to_none=True)
            m(x, o).backward(g)
    torch.cuda.current_stream().wait_stream(s)
    m.zero_grad(set_to_none=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gw, gb = torch.autograd.grad(m(x, o), [m.weight, m.bias], g)
    alive = m(x, o)  # an eager graph of the same leaves
    for i in range(3):
        graph.replay()
        torch.cuda.synchronize()
        ew, eb = torch.autograd.grad(m(x, o), [m.weight, m.bias], g)
        torch.cuda.synchronize()
        assert torch.equal(gw, ew) and torch.equal(gb, eb), i
    alive.backward(g)
    assert torch.equal(m.weight.grad, ew)


def test_other_current_device_is_not_needed():
    """The calls run on the tensors' device and refuse a stream of another."""
    x = bf16((4, 64), 1.0, 1).to(DEV)
    q, s = torch.empty(4, 64, dtype=torch.int8, device=DEV), torch.empty(4, device=DEV)

    class Other:
        device = torch.device("cuda", 1)
        cuda_stream = 0

    with pytest.raises(ValueError, match="stream"):
        F.fp8_i8_quantize_rows(x, q, s, stream=Other())
