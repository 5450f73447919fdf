"""Row-wise 8-bit integer quantize and the integer linear layers on the GPU:
codes and scales bit for bit against the oracle, outputs within the bound
that the arithmetic allows, exact cases bit for bit."""

import numpy as np
import pytest
import torch

import scaled_quantize_fp8_amd as F
from oracle import rows_oracle as R
from tests.gpu_util import DEV, f32, to_dev
from tests.rows_util import GROUPS, bf16, check_i8, offsets_dev, offsets_of, outside

pytestmark = pytest.mark.gpu

TILES = ["v1", "128x128w8", "256x256w8", "128x256", "skinny16", "skinny32",
         "skinny48", "skinny64", None]
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _tile(monkeypatch, tile):
    if tile is None:
        monkeypatch.delenv("FP8L_TILE", raising=False)
    else:
        monkeypatch.setenv("FP8L_TILE", tile)


def _x(rows, cols, dt, seed=1):
    rng = np.random.default_rng(seed)
    v = rng.standard_normal((rows, cols)) * 10.0 ** rng.uniform(-2, 2, (rows, 1))
    return torch.from_numpy(v).to(DT[dt])


def _weights(shape, seed=2):
    rng = np.random.default_rng(seed)
    return (rng.integers(-127, 128, shape).astype(np.int8),
            np.float32(rng.uniform(20, 5000, shape[:-1])))


def _quantize(x):
    q = torch.full(x.shape, 99, dtype=torch.int8, device=DEV)
    s = torch.empty(x.shape[:-1], dtype=torch.float32, device=DEV)
    F.fp8_i8_quantize_rows(x.to(DEV), q, s)
    return q.cpu().numpy(), s.cpu().numpy()


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (1, 4096), (5, 8), (300, 264), (17, 1031),
                                       (2, 16384), (2100, 64), (4, 20001), (9, 2048), (7, 33000)])
def test_quantize_rows_bit_exact(rows, cols, dt):
    x = _x(rows, cols, dt)
    q, s = _quantize(x)
    oq, os = R.i8_quantize_rows(f32(x))
    assert np.array_equal(s, os) and np.array_equal(q, oq)


@pytest.mark.parametrize("dt", list(DT))
def test_quantize_rows_specials(dt):
    """Zero rows, a NaN, infinities, subnormals, the largest values, ties."""
    big = torch.finfo(DT[dt]).max
    tiny = torch.finfo(DT[dt]).tiny / 4  # subnormal
    rows = [[0.0] * 9, [1.0, float("nan")] + [2.0] * 7, [float("inf")] + [1.0] * 8,
            [1.0] * 8 + [float("-inf")], [big, -big, big / 2] + [0.0] * 6,
            [tiny, -tiny, tiny * 0.5] + [0.0] * 6, [127.0, 0.5, 1.5, -2.5, 126.5] + [0.0] * 4,
            [-0.0] * 9, [1.0] * 9]
    for width in (9, 16, 1000):
        x = torch.zeros(len(rows), width, dtype=torch.float64)
        x[:, :9] = torch.tensor(rows, dtype=torch.float64)
        x = x.to(DT[dt])
        q, s = _quantize(x)
        oq, os = R.i8_quantize_rows(f32(x))
        assert np.array_equal(s, os, equal_nan=True) and np.array_equal(q, oq)


def test_quantize_rows_leading_dims_and_empty():
    x = _x(12, 40, "bf16").view(3, 4, 40)
    q, s = _quantize(x)
    oq, os = R.i8_quantize_rows(f32(x).reshape(12, 40))
    assert np.array_equal(q.reshape(12, 40), oq) and np.array_equal(s.reshape(12), os)
    _quantize(torch.empty(0, 40, dtype=torch.bfloat16))
    _, s = _quantize(torch.empty(4, 0, dtype=torch.bfloat16))
    assert (s == 1).all()


def test_quantize_rows_unaligned_pointer():
    base = _x(1, 8 * 200 + 1, "bf16").reshape(-1)
    x = base[1:].view(8, 200)
    q, s = torch.empty(8 * 200 + 3, dtype=torch.int8, device=DEV), torch.empty(8, device=DEV)
    F.fp8_i8_quantize_rows(base.to(DEV)[1:].view(8, 200), q[3:].view(8, 200), s)
    oq, os = R.i8_quantize_rows(f32(x))
    assert np.array_equal(q[3:].view(8, 200).cpu().numpy(), oq)
    assert np.array_equal(s.cpu().numpy(), os)


def _linear(M, N, K, dt, out, bias, seed=5):
    x = _x(M, K, dt, seed) if M * K else torch.empty(M, K, dtype=DT[dt])
    w, sw = _weights((N, K), seed + 1)
    b = None if not bias else (bf16((N,), 2.0, seed + 2)).to(DT[out])
    y = torch.full((M, N), 7.0, dtype=DT[out], device=DEV)
    x8, sx = torch.empty(M, K, dtype=torch.int8, device=DEV), torch.empty(M, device=DEV)
    F.fp8_i8_linear_fwd(x.to(DEV), F.QuantizedRows(to_dev(w), to_dev(sw)),
                        None if b is None else b.to(DEV), y, x8, sx)
    oq, os = R.i8_quantize_rows(f32(x))
    assert np.array_equal(x8.cpu().numpy(), oq) and np.array_equal(sx.cpu().numpy(), os)
    r, p = R.i8_linear(oq, os, w, sw, None if b is None else f32(b))
    check_i8(y, r, p, out, f"{M}x{N}x{K}")


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("M,N,K", [(1, 64, 64), (129, 136, 96), (256, 256, 4096), (300, 520, 208),
                                   (64, 64, 0)])
@pytest.mark.parametrize("out,bias", [("bf16", True), ("fp16", False), ("fp16", True)])
def test_linear_tiles(M, N, K, out, bias, tile, monkeypatch):
    _tile(monkeypatch, tile)
    _linear(M, N, K, "bf16", out, bias)


@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8, 9, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 100])
@pytest.mark.parametrize("N,K", [(64, 128), (1000, 4096), (200, 11008)])
def test_linear_few_rows(M, N, K):
    _linear(M, N, K, "bf16", "bf16", True)


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (3, 5, 7), (16, 33, 1003), (70, 777, 130),
                                   (129, 1, 40), (5, 131, 48), (2, 200, 24)])
@pytest.mark.parametrize("dt,out", [("fp32", "bf16"), ("fp16", "fp16")])
def test_linear_odd_sizes(M, N, K, dt, out):
    _linear(M, N, K, dt, out, True)


def test_linear_empty():
    _linear(0, 16, 16, "bf16", "bf16", True)
    _linear(4, 0, 16, "bf16", "bf16", False)


@pytest.mark.parametrize("M", [1, 20, 200])
@pytest.mark.parametrize("tile", TILES)
def test_sums_are_exact_at_the_largest_codes(M, tile, monkeypatch):
    """All codes at +-127 (and -128 in the weights) over a long contraction,
    scales powers of two: the output is the correctly rounded exact sum."""
    _tile(monkeypatch, tile)
    N, K = 80, 131056
    rng = np.random.default_rng(8)
    q = rng.choice(np.int8([-127, 127]), (M, K))
    w = rng.choice(np.int8([-128, 127]), (N, K))
    q[0], w[0], w[1] = 127, 127, -128  # the largest sums of either sign
    y = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    F.fp8_i8_linear_fwd(F.QuantizedRows(to_dev(q), torch.full((M,), 4.0, device=DEV)),
                        F.QuantizedRows(to_dev(w), torch.full((N,), 0.5, device=DEV)), None, y)
    want = torch.from_numpy((q.astype(np.float64) @ w.astype(np.float64).T) * 0.5)
    # sums beyond 2^24 round once to fp32 and once to bf16, as the kernel does
    assert torch.equal(y.cpu(), want.to(torch.float32).to(torch.bfloat16))


def test_nonfinite_token_stays_alone():
    M, N, K = 40, 96, 128
    x = _x(M, K, "bf16")
    x[3, 5], x[17, 0] = float("nan"), float("inf")
    w, sw = _weights((N, K))
    y = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    F.fp8_i8_linear_fwd(x.to(DEV), F.QuantizedRows(to_dev(w), to_dev(sw)), None, y,
                        torch.empty(M, K, dtype=torch.int8, device=DEV),
                        torch.empty(M, device=DEV))
    oq, os = R.i8_quantize_rows(f32(x))
    r, p = R.i8_linear(oq, os, w, sw)
    assert np.isnan(r[[3, 17]]).all() and np.isfinite(np.delete(r, [3, 17], 0)).all()
    check_i8(y, r, p, "bf16")


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("name", list(GROUPS))
@pytest.mark.parametrize("N,K,out,bias", [(96, 144, "bf16", True), (272, 64, "fp16", False),
                                          (33, 50, "bf16", True)])
def test_grouped(name, N, K, out, bias, tile, monkeypatch):
    _tile(monkeypatch, tile)
    T, off = offsets_of(name)
    E = len(off) - 1
    x = _x(T, K, "bf16")
    x[torch.from_numpy(outside(T, off))] = float("nan")
    w, sw = _weights((E, N, K))
    b = bf16((E, N), 2.0, 3).to(DT[out]) if bias else None
    y = torch.full((T, N), 7.0, dtype=DT[out], device=DEV)
    x8 = torch.full((T, K), 99, dtype=torch.int8, device=DEV)
    sx = torch.full((T,), -1.0, device=DEV)
    F.fp8_i8_grouped_linear_fwd(x.to(DEV), F.QuantizedRows(to_dev(w), to_dev(sw)),
                                None if b is None else b.to(DEV), offsets_dev(off), y, x8, sx)
    oq, os = R.i8_quantize_rows(f32(x))
    for e, i, j in R.spans(off):
        if i < j:
            r, p = R.i8_linear(oq[i:j], os[i:j], w[e], sw[e], None if b is None else f32(b)[e])
            check_i8(y[i:j], r, p, out, f"group {e}")
    used = off[-1]
    assert (y.cpu()[torch.from_numpy(outside(T, off))] == 7.0).all()
    assert (x8[used:] == 99).all() and (sx[used:] == -1).all()


@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("M", [1, 24, 300])
def test_captured_call_replays_like_eager_ones(M, grouped):
    N, K, E = 160, 512, 5
    w, sw = _weights((E, N, K) if grouped else (N, K))
    W = F.QuantizedRows(to_dev(w), to_dev(sw))
    x = _x(M, K, "bf16").to(DEV)
    offs = [offsets_dev([0, M // 3, M // 3, M // 2, M, M]), offsets_dev([0, 0, M, M, M, M])]
    off = offs[0].clone()
    y, y2 = (torch.empty(M, N, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    x8, sx = torch.empty(M, K, dtype=torch.int8, device=DEV), torch.empty(M, device=DEV)

    def run(out):
        if grouped:
            F.fp8_i8_grouped_linear_fwd(x, W, None, off, out, x8, sx)
        else:
            F.fp8_i8_linear_fwd(x, W, None, out, x8, sx)

    run(y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(y)
    for i in range(4):
        x.copy_(_x(M, K, "bf16", seed=40 + i))
        off.copy_(offs[i % 2])
        y.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        run(y2)
        torch.cuda.synchronize()
        assert torch.equal(y, y2)


def test_calls_on_several_streams():
    M, N, K = 65, 304, 1024
    w, sw = _weights((N, K))
    W = F.QuantizedRows(to_dev(w), to_dev(sw))
    xs = [_x(M, K, "bf16", seed=50 + i).to(DEV) for i in range(4)]

    def buffers():
        return (torch.empty(M, N, dtype=torch.bfloat16, device=DEV),
                torch.empty(M, K, dtype=torch.int8, device=DEV), torch.empty(M, device=DEV))

    want = []
    for x in xs:
        y, q, s = buffers()
        F.fp8_i8_linear_fwd(x, W, None, y, q, s)
        want.append(y)
    outs = [buffers() for _ in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, x, (y, q, sc) in zip(streams, xs, outs):
            F.fp8_i8_linear_fwd(x, W, None, y, q, sc, stream=s)
    torch.cuda.synchronize()
    for (y, _, _), v in zip(outs, want):
        assert torch.equal(y, v)


def test_rows_beyond_one_buffer_resource():
    """X codes of more than 2^31 bytes: the first and the last rows against
    the oracle (the tiles move their own rows into reach)."""
    M, N, K = 150_000, 64, 14_400
    w, sw = _weights((N, K))
    x8 = torch.zeros(M, K, dtype=torch.int8, device=DEV)
    sx = torch.ones(M, device=DEV)
    rows = [0, 1, M // 2, M - 130, M - 1]
    q = np.random.default_rng(3).integers(-127, 128, (len(rows), K)).astype(np.int8)
    x8[torch.tensor(rows, device=DEV)] = to_dev(q)
    y = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    F.fp8_i8_linear_fwd(F.QuantizedRows(x8, sx), F.QuantizedRows(to_dev(w), to_dev(sw)), None, y)
    r, p = R.i8_linear(q, np.ones(len(rows), np.float32), w, sw)
    check_i8(y[torch.tensor(rows, device=DEV)], r, p, "bf16")
    assert not y[M - 129:M - 1].any() and not y[2:M // 2].any()


@pytest.mark.parametrize("dt,out", [("bf16", "bf16"), ("fp16", "fp16"), ("fp32", "bf16")])
@pytest.mark.parametrize("M,N,K", [(1, 64, 16), (1, 4096, 4096), (2, 1000, 1040), (3, 72, 16384),
                                   (4, 136, 11008), (4, 8, 144)])
def test_few_rows_quantized_in_the_product_launch(M, N, K, dt, out):
    _linear(M, N, K, dt, out, True)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("K", [32, 1536, 4096])
def test_grouped_few_rows_of_every_type(K, dt):
    """Codes, scales and outputs of groups of up to 20 rows, a NaN token and a
    zero token among them, quantized inside the product's launch."""
    N = 72
    T, off = offsets_of("few")
    E = len(off) - 1
    assert T <= 2 * E
    x = _x(T, K, dt)
    x[3, 5] = float("nan")
    x[21] = 0
    w, sw = _weights((E, N, K))
    y = torch.full((T, N), 7.0, dtype=torch.bfloat16, device=DEV)
    x8 = torch.full((T, K), 99, dtype=torch.int8, device=DEV)
    sx = torch.full((T,), -1.0, device=DEV)
    F.fp8_i8_grouped_linear_fwd(x.to(DEV), F.QuantizedRows(to_dev(w), to_dev(sw)), None,
                                offsets_dev(off), y, x8, sx)
    oq, os = R.i8_quantize_rows(f32(x))
    used = off[-1]
    assert np.array_equal(x8.cpu().numpy()[:used], oq[:used])
    assert np.array_equal(sx.cpu().numpy()[:used], os[:used], equal_nan=True)
    assert (x8[used:] == 99).all() and (sx[used:] == -1).all() and (y[used:] == 7.0).all()
    for e, i, j in R.spans(off):
        if i < j:
            r, p = R.i8_linear(oq[i:j], os[i:j], w[e], sw[e])
            check_i8(y[i:j], r, p, "bf16", f"group {e}")


@pytest.mark.parametrize("T,K", [(1, 16384), (2, 4096), (2, 4112), (4, 512)])
def test_one_expert(T, K):
    """A single group: the grouped call equals the dense one bit for bit."""
    N = 80
    x = _x(T, K, "bf16").to(DEV)
    w, sw = _weights((1, N, K))
    W, off = to_dev(w), offsets_dev([0, T])
    y, z = (torch.empty(T, N, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    q, s = torch.empty(T, K, dtype=torch.int8, device=DEV), torch.empty(T, device=DEV)
    F.fp8_i8_grouped_linear_fwd(x, F.QuantizedRows(W, to_dev(sw)), None, off, y, q, s)
    F.fp8_i8_linear_fwd(x, F.QuantizedRows(W[0], to_dev(sw[0])), None, z, q, s)
    assert torch.equal(y, z)


def test_a_grid_larger_than_2_to_the_32_threads():
    """2^30 output channels of one weight each: the tile that few rows take
    would need 2^32 threads, so the general one runs."""
    N = (1 << 30) + 5
    i = torch.arange(N, dtype=torch.int32, device=DEV)
    w = (i % 251 - 125).to(torch.int8)
    sw = torch.full((N,), 0.5, device=DEV)
    y = torch.full((1, N), 7.0, dtype=torch.bfloat16, device=DEV)
    F.fp8_i8_linear_fwd(F.QuantizedRows(torch.full((1, 1), 3, dtype=torch.int8, device=DEV),
                                        torch.full((1,), 2.0, device=DEV)),
                        F.QuantizedRows(w.view(N, 1), sw), None, y)
    # 3 w / (2 * 0.5): at most 375, rounded once
    for c in range(0, N, 1 << 28):
        assert torch.equal(y[0, c:c + (1 << 28)], (3 * w[c:c + (1 << 28)].float()).to(torch.bfloat16))
