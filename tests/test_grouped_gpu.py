"""The FP8 linear layers over ragged groups of rows on the GPU against the
oracle, group by group: every tile kernel and the general one, group sizes
at the tile edges, empty groups, rows of no group, all format pairs, the
quantizing calls with rings and dynamic scales, graphs, streams, repeats."""

import numpy as np
import pytest
import torch

import scaled_quantize_fp8_amd as F
from oracle import fp8_oracle as O
from oracle import rows_oracle as R
from tests.gpu_util import (DEV, assert_ring_matches, bf16_bits, check_gemm, f32, f32_scalar,
                            scalar_dev, to_dev, u8)
from tests.rows_util import (GROUPS, bf16, check_groups, offsets_dev, offsets_of, outside,
                             random_codes)

pytestmark = pytest.mark.gpu

TILES = ["v1", "128x128w8", "256x256w8", "128x256", "skinny16", "skinny32",
         "skinny48", "skinny64", None]
SENTINEL = 7.0


def _tile(monkeypatch, tile):
    if tile is None:
        monkeypatch.delenv("FP8L_TILE", raising=False)
    else:
        monkeypatch.setenv("FP8L_TILE", tile)


def _operands(name, N, K, fmt_x=O.E4M3, fmt_w=O.E4M3, seed=1, per_expert=True):
    T, off = offsets_of(name)
    E = len(off) - 1
    x8, w8 = random_codes((T, K), seed, fmt_x), random_codes((E, N, K), seed + 1, fmt_w)
    rng = np.random.default_rng(seed + 2)
    sx = np.float32(rng.uniform(0.5, 4))
    sw = np.float32(rng.uniform(0.5, 4, E if per_expert else 1))
    return T, off, E, x8, w8, sx, sw


def _filled(*shape):
    return torch.full(shape, SENTINEL, dtype=torch.bfloat16, device=DEV)


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("name", list(GROUPS))
@pytest.mark.parametrize("N,K,bias", [(96, 144, True), (272, 64, False)])
def test_forward(name, N, K, bias, tile, monkeypatch):
    _tile(monkeypatch, tile)
    T, off, E, x8, w8, sx, sw = _operands(name, N, K)
    b = bf16((E, N), 1.0, 9) if bias else None
    y = _filled(T, N)
    F.fp8_grouped_linear_fwd(F.Quantized(to_dev(x8), O.E4M3, scalar_dev(sx)),
                             F.Quantized(to_dev(w8), O.E4M3, to_dev(sw)),
                             None if b is None else b.to(DEV), offsets_dev(off), O.E4M3, y)
    refs = R.grouped_fwd(x8, w8, O.E4M3, sx, sw, off, None if b is None else f32(b).astype(float))
    check_groups(y, refs, off, "y")
    assert (y.cpu()[torch.from_numpy(outside(T, off))] == SENTINEL).all()


@pytest.mark.parametrize("N,K", [(1, 1), (5, 3), (33, 130), (130, 33), (96, 40), (24, 48)])
@pytest.mark.parametrize("fmt", [O.E4M3, O.E5M2])
def test_forward_odd_sizes(N, K, fmt):
    T, off, E, x8, w8, sx, sw = _operands("edges", N, K, fmt, fmt, per_expert=False)
    b = bf16((E, N), 1.0, 9)
    y = _filled(T, N)
    F.fp8_grouped_linear_fwd(F.Quantized(to_dev(x8), fmt, scalar_dev(sx)),
                             F.Quantized(to_dev(w8), fmt, to_dev(sw)), b.to(DEV),
                             offsets_dev(off), fmt, y)
    check_groups(y, R.grouped_fwd(x8, w8, fmt, sx, sw, off, f32(b).astype(float)), off, "y")


@pytest.mark.parametrize("tile", TILES)
def test_forward_without_contraction_is_the_bias(tile, monkeypatch):
    _tile(monkeypatch, tile)
    T, off = offsets_of("tail")
    E, N = len(off) - 1, 64
    b = bf16((E, N), 1.0, 9)
    y = _filled(T, N)
    F.fp8_grouped_linear_fwd(
        F.Quantized(torch.empty(T, 0, dtype=torch.uint8, device=DEV), O.E4M3, scalar_dev(1)),
        F.Quantized(torch.empty(E, N, 0, dtype=torch.uint8, device=DEV), O.E4M3, scalar_dev(1)),
        b.to(DEV), offsets_dev(off), O.E4M3, y)
    for e, i, j in R.spans(off):
        assert (y[i:j].cpu() == b[e]).all()


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("name", list(GROUPS))
@pytest.mark.parametrize("N,K", [(96, 144), (272, 64)])
def test_backward(name, N, K, tile, monkeypatch):
    """dX, dW and db from pre-quantized operands (G in e5m2)."""
    _tile(monkeypatch, tile)
    T, off, E, x8, w8, sx, sw = _operands(name, N, K)
    g8, sg = random_codes((T, N), 5, O.E5M2), np.float32(3.0)
    dx, dw, db = _filled(T, K), _filled(E, N, K), _filled(E, N)
    ws = torch.empty(F.fp8_grouped_db_workspace_bytes(T, E, N), dtype=torch.uint8, device=DEV)
    F.fp8_grouped_linear_bwd(F.Quantized(to_dev(g8), O.E5M2, scalar_dev(sg)), O.E5M2,
                             offsets_dev(off), F.Quantized(to_dev(x8), O.E4M3, scalar_dev(sx)),
                             F.Quantized(to_dev(w8), O.E4M3, to_dev(sw)), dx, dw, db, ws)
    check_groups(dx, R.grouped_dx(g8, O.E5M2, w8, O.E4M3, sg, sw, off), off, "dx")
    assert (dx.cpu()[torch.from_numpy(outside(T, off))] == SENTINEL).all()
    dbs = R.grouped_db(O.dequantized(g8, O.E5M2, sg), off)
    for e, ref in enumerate(R.grouped_dw(g8, O.E5M2, x8, O.E4M3, sg, sx, off)):
        if ref is None:
            assert not dw[e].any() and not db[e].any()
        else:
            check_gemm(bf16_bits(dw[e]), ref, f"dw {e}")
            check_gemm(bf16_bits(db[e]), dbs[e], f"db {e}")


@pytest.mark.parametrize("N,K", [(1, 1), (5, 3), (33, 130), (96, 40), (40, 96)])
@pytest.mark.parametrize("fg", [O.E4M3, O.E5M2])
@pytest.mark.parametrize("fw", [O.E4M3, O.E5M2])
def test_backward_odd_sizes_and_formats(N, K, fg, fw):
    T, off, E, x8, w8, sx, sw = _operands("edges", N, K, fw, fw)
    g8, sg = random_codes((T, N), 5, fg), np.float32(3.0)
    dx, dw, db = _filled(T, K), _filled(E, N, K), _filled(E, N)
    ws = torch.empty(F.fp8_grouped_db_workspace_bytes(T, E, N), dtype=torch.uint8, device=DEV)
    F.fp8_grouped_linear_bwd(F.Quantized(to_dev(g8), fg, scalar_dev(sg)), fg, offsets_dev(off),
                             F.Quantized(to_dev(x8), fw, scalar_dev(sx)),
                             F.Quantized(to_dev(w8), fw, to_dev(sw)), dx, dw, db, ws)
    check_groups(dx, R.grouped_dx(g8, fg, w8, fw, sg, sw, off), off, "dx")
    dbs = R.grouped_db(O.dequantized(g8, fg, sg), off)
    for e, ref in enumerate(R.grouped_dw(g8, fg, x8, fw, sg, sx, off)):
        if ref is not None:
            check_gemm(bf16_bits(dw[e]), ref, f"dw {e}")
            check_gemm(bf16_bits(db[e]), dbs[e], f"db {e}")


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("hist", [None, 16, 100])
def test_quantizing_steps_match_the_oracle(dt, hist):
    """Two training steps from high-precision X, W and G, rows behind the last
    group holding NaN: codes, scales, amax and rings equal the oracle's on the
    rows in use; outputs equal the grouped GEMMs of those codes."""
    N, K = 80, 112
    T, off = offsets_of("tail")
    E, used = len(off) - 1, off[-1]
    rings = [None] * 3 if hist is None else [F.ScaleRing(hist) for _ in range(3)]
    orings = [None] * 3 if hist is None else [O.ScaleRing(hist) for _ in range(3)]
    f = lambda: torch.empty(1, dtype=torch.float32, device=DEV)
    for step in range(2):
        X, W, G = ((bf16(sh, s * (1 + 3 * step), 20 + i).to(dt))
                   for i, (sh, s) in enumerate((((T, K), 1.0), ((E, N, K), 0.02), ((T, N), 1e-2))))
        X[used:] = float("nan")
        G[used:] = float("nan")
        x8, w8, g8 = (torch.full(s, 0xAA, dtype=torch.uint8, device=DEV)
                      for s in ((T, K), (E, N, K), (T, N)))
        sx, sw, sg, ax, aw, ag = (f() for _ in range(6))
        y, dx, dw, db = _filled(T, N), _filled(T, K), _filled(E, N, K), _filled(E, N)
        F.fp8_grouped_linear_fwd(X.to(DEV), W.to(DEV), None, offsets_dev(off), O.E4M3, y, rings[0],
                                 rings[1], x8, w8, sx, sw, ax, aw)
        ws = torch.full((F.fp8_grouped_db_workspace_bytes(T, E, N),), 0xFF, dtype=torch.uint8,
                        device=DEV)
        F.fp8_grouped_linear_bwd(G.to(DEV), O.E5M2, offsets_dev(off),
                                 F.Quantized(x8, O.E4M3, sx), F.Quantized(w8, O.E4M3, sw), dx, dw,
                                 db, ws, rings[2], g8, sg, ag)
        ox, osx, oax = O.quantize_step(f32(X)[:used], O.E4M3, orings[0])
        ow, osw, oaw = O.quantize_step(f32(W), O.E4M3, orings[1])
        og, osg, oag = O.quantize_step(f32(G)[:used], O.E5M2, orings[2])
        for got, want in ((x8, ox), (w8, ow), (g8, og)):
            assert np.array_equal(u8(got)[:len(want)], want)
        assert (u8(x8)[used:] == 0xAA).all() and (u8(g8)[used:] == 0xAA).all()
        for got, want in ((sx, osx), (sw, osw), (sg, osg), (ax, oax), (aw, oaw), (ag, oag)):
            assert f32_scalar(got) == np.float32(want)
        if hist is not None:
            for r, o in zip(rings, orings):
                assert_ring_matches(r, o)
        check_groups(y, R.grouped_fwd(ox, ow, O.E4M3, osx, [osw], off), off, "y")
        check_groups(dx, R.grouped_dx(og, O.E5M2, ow, O.E4M3, osg, [osw], off), off, "dx")
        dbs = R.grouped_db(f32(G)[:used].astype(np.float64), off)
        for e, ref in enumerate(R.grouped_dw(og, O.E5M2, ox, O.E4M3, osg, osx, off)):
            if ref is not None:
                check_gemm(bf16_bits(dw[e]), ref, f"dw {e}")
                check_gemm(bf16_bits(db[e]), dbs[e], f"db {e}")


@pytest.mark.parametrize("want", ["dx", "dw", "db"])
def test_single_gradients(want):
    """Each gradient alone equals the full call's, with a ring on G."""
    N, K = 96, 144
    T, off, E, x8, w8, sx, sw = _operands("edges", N, K)
    G = bf16((T, N), 1e-3, 4).to(DEV)
    X, W = F.Quantized(to_dev(x8), O.E4M3, scalar_dev(sx)), F.Quantized(to_dev(w8), O.E4M3,
                                                                       to_dev(sw))
    ws = torch.empty(F.fp8_grouped_db_workspace_bytes(T, E, N), dtype=torch.uint8, device=DEV)

    def call(names, ring):
        out = {"dx": _filled(T, K), "dw": _filled(E, N, K), "db": _filled(E, N)}
        given = {k: (v if k in names else None) for k, v in out.items()}
        F.fp8_grouped_linear_bwd(G, O.E5M2, offsets_dev(off), X if "dw" in names else None,
                                 W if "dx" in names else None, given["dx"], given["dw"],
                                 given["db"], ws if "db" in names else None, ring,
                                 torch.empty(T, N, dtype=torch.uint8, device=DEV),
                                 torch.empty(1, device=DEV))
        return out

    full, alone = F.ScaleRing(16), F.ScaleRing(16)
    for _ in range(2):  # the seeding step and a steady one
        a, b = call(("dx", "dw", "db"), full), call((want,), alone)
        assert torch.equal(a[want], b[want])
        for k in b:
            if k != want:
                assert (b[k] == SENTINEL).all()
        assert torch.equal(full.buf, alone.buf)


def test_scales_of_quantized_operands_are_snapshotted():
    N, K = 32, 32
    T, off, E, x8, w8, sx, sw = _operands("edges", N, K)
    out = [torch.full((n,), -1.0, device=DEV) for n in (1, E, 1, 1)]
    F.fp8_grouped_linear_fwd(F.Quantized(to_dev(x8), O.E4M3, scalar_dev(sx)),
                             F.Quantized(to_dev(w8), O.E4M3, to_dev(sw)), None, offsets_dev(off),
                             O.E4M3, _filled(T, N), sx_used=out[0], sw_used=out[1], amax_x=out[2],
                             amax_w=out[3])
    assert f32_scalar(out[0]) == sx and np.array_equal(out[1].cpu().numpy(), sw)
    assert out[2].item() == 0 and out[3].item() == 0


def _step(T, off, E, N, K, X, W, G, rings, b):
    f = lambda: torch.empty(1, dtype=torch.float32, device=DEV)
    u = lambda *s: torch.empty(*s, dtype=torch.uint8, device=DEV)
    buf = dict(y=_filled(T, N), dx=_filled(T, K), dw=_filled(E, N, K), db=_filled(E, N),
               x8=u(T, K), w8=u(E, N, K), g8=u(T, N), sx=f(), sw=f(), sg=f(), am=[f(), f(), f()],
               ws=u(F.fp8_grouped_db_workspace_bytes(T, E, N)), off=offsets_dev(off))

    def run():
        F.fp8_grouped_linear_fwd(X, W, b, buf["off"], O.E4M3, buf["y"], rings[0], rings[1],
                                 buf["x8"], buf["w8"], buf["sx"], buf["sw"], *buf["am"][:2])
        F.fp8_grouped_linear_bwd(G, O.E5M2, buf["off"], F.Quantized(buf["x8"], O.E4M3, buf["sx"]),
                                 F.Quantized(buf["w8"], O.E4M3, buf["sw"]), buf["dx"], buf["dw"],
                                 buf["db"], buf["ws"], rings[2], buf["g8"], buf["sg"],
                                 buf["am"][2])
    return buf, run


@pytest.mark.parametrize("dynamic", [False, True])
def test_captured_steps_replay_like_eager_ones(dynamic):
    """A forward and backward captured into a graph: replays with new inputs
    and new offsets, eager work between them, equal eager calls bit for bit."""
    N, K = 96, 144
    T, off = offsets_of("edges")
    E = len(off) - 1
    other = [0, 100, 100, 110, 110, 300, 500, 600, 640, T]
    X, W, G = (bf16(s, 1.0, 30 + i).to(DEV) for i, s in enumerate(((T, K), (E, N, K), (T, N))))
    b = bf16((E, N), 1.0, 33).to(DEV)
    rings, erings = ([None] * 3 if dynamic else [F.ScaleRing(16) for _ in range(3)]
                     for _ in range(2))
    buf, run = _step(T, off, E, N, K, X, W, G, rings, b)
    ebuf, erun = _step(T, off, E, N, K, X, W, G, erings, b)
    run(), erun()  # seeds the rings
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for i in range(4):
        X.mul_(1.5)
        G.mul_(0.75)
        o = offsets_dev(other if i % 2 else off)
        buf["off"].copy_(o)
        ebuf["off"].copy_(o)
        for k in ("y", "dx", "dw", "db"):
            buf[k].fill_(SENTINEL)
            ebuf[k].fill_(SENTINEL)
        graph.replay()
        torch.cuda.synchronize()
        erun()
        torch.cuda.synchronize()
        for k in ("y", "dx", "dw", "db"):
            assert torch.equal(buf[k], ebuf[k]), (i, k)
        for k in ("x8", "g8", "sx", "sg"):
            assert torch.equal(buf[k], ebuf[k]), (i, k)


def test_unseeded_ring_is_refused_under_capture():
    N, K = 32, 32
    T, off = offsets_of("one")
    X, W, G = (bf16(s, 1.0, 30 + i).to(DEV) for i, s in enumerate(((T, K), (1, N, K), (T, N))))
    rings = [F.ScaleRing(16) for _ in range(3)]
    buf, run = _step(T, off, 1, N, K, X, W, G, rings, None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(F.Fp8Error) as err:
        with torch.cuda.graph(graph):
            run()
    assert err.value.status == F.FP8_ERR_RING and not rings[0].seeded


def test_repeated_calls_give_the_same_bits_on_other_streams():
    N, K = 272, 144
    T, off = offsets_of("edges")
    E = len(off) - 1
    X, W, G = (bf16(s, 1.0, 30 + i).to(DEV) for i, s in enumerate(((T, K), (E, N, K), (T, N))))
    buf, run = _step(T, off, E, N, K, X, W, G, [None] * 3, None)
    run()
    torch.cuda.synchronize()
    want = {k: buf[k].clone() for k in ("y", "dx", "dw", "db")}
    streams = [torch.cuda.Stream() for _ in range(3)]
    runs = [_step(T, off, E, N, K, X, W, G, [None] * 3, None) for _ in streams]
    torch.cuda.synchronize()
    for s, (_, r) in zip(streams, runs):
        with torch.cuda.stream(s):
            for _ in range(5):
                r()
    torch.cuda.synchronize()
    for bb, _ in runs:
        for k, v in want.items():
            assert torch.equal(bb[k], v), k


def test_wild_offsets_stay_inside_the_operands():
    """Offsets past T or decreasing are clamped: guard rows around the outputs
    keep their values."""
    N, K, T = 64, 64, 100
    x8, w8 = random_codes((T, K), 1, O.E4M3), random_codes((3, N, K), 2, O.E4M3)
    big = _filled(T + 512, N)
    y = big[256:256 + T]
    off = torch.tensor([-5, 60, 20, 1 << 30], dtype=torch.int32, device=DEV)
    F.fp8_grouped_linear_fwd(F.Quantized(to_dev(x8), O.E4M3, scalar_dev(1)),
                             F.Quantized(to_dev(w8), O.E4M3, scalar_dev(1)), None, off, O.E4M3, y)
    torch.cuda.synchronize()
    assert (big[:256] == SENTINEL).all() and (big[256 + T:] == SENTINEL).all()


def test_small_dynamic_quantize_matches_the_general_one():
    """The one-launch quantize of a small G gives the codes, scale and amax of
    the amax-pass form (the same G in front of rows of no group)."""
    N, K = 64, 48
    T, off = offsets_of("tail")
    E, used = len(off) - 1, off[-1]
    G = bf16((T, N), 1e-2, 5)
    big = torch.zeros(2048, N, dtype=torch.bfloat16)
    big[:T] = G
    big[used:] = float("nan")
    out = []
    for g in (G, big):
        rows = g.shape[0]
        g8 = torch.zeros(rows, N, dtype=torch.uint8, device=DEV)
        sg, am = torch.empty(1, device=DEV), torch.empty(1, device=DEV)
        db = _filled(E, N)
        ws = torch.empty(F.fp8_grouped_db_workspace_bytes(rows, E, N), dtype=torch.uint8,
                         device=DEV)
        F.fp8_grouped_linear_bwd(g.to(DEV), O.E5M2, offsets_dev(off), None, None, db=db, db_ws=ws,
                                 g8_out=g8, sg_used=sg, amax_g=am)
        out.append((g8[:used].cpu(), sg.cpu(), am.cpu(), db.cpu()))
    assert T * N <= 65536 < 2048 * N
    for a, b in zip(*out):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dt,N", [(torch.bfloat16, 80), (torch.float32, 33)])
@pytest.mark.parametrize("hist", [None, 16, 100])
@pytest.mark.parametrize("front", [1, 32, 45])
def test_rows_before_the_first_group_are_quantized(front, hist, dt, N):
    """G over [0, offsets[E]), its largest value before the first group: codes,
    scale, amax and ring are the oracle's with db and without it (in two
    steps), and no sum holds those rows."""
    off, T, K = [front, front + 16, front + 16, front + 49], front + 58, 32
    E, used = len(off) - 1, off[-1]
    x8, w8 = random_codes((T, K), 1, O.E4M3), random_codes((E, N, K), 2, O.E4M3)
    for with_db in (True, False):
        ring = None if hist is None else F.ScaleRing(hist)
        oring = None if hist is None else O.ScaleRing(hist)
        for step in range(2):
            G = bf16((T, N), 1e-2 * (1 + step), 30 + step).to(dt)
            G[front - 1, N // 2] = 0.5 + step
            G[used:] = float("nan")
            g8 = torch.full((T, N), 0xAA, dtype=torch.uint8, device=DEV)
            sg, ag = (torch.empty(1, dtype=torch.float32, device=DEV) for _ in range(2))
            dw = _filled(E, N, K)
            db = _filled(E, N) if with_db else None
            ws = torch.full((F.fp8_grouped_db_workspace_bytes(T, E, N),), 0xFF, dtype=torch.uint8,
                            device=DEV)
            F.fp8_grouped_linear_bwd(G.to(DEV), O.E5M2, offsets_dev(off),
                                     F.Quantized(to_dev(x8), O.E4M3, scalar_dev(1)),
                                     F.Quantized(to_dev(w8), O.E4M3, scalar_dev(1)), None, dw, db,
                                     ws, ring, g8, sg, ag)
            og, osg, oag = O.quantize_step(f32(G)[:used], O.E5M2, oring)
            assert np.array_equal(u8(g8)[:used], og) and (u8(g8)[used:] == 0xAA).all()
            assert f32_scalar(sg) == np.float32(osg) and f32_scalar(ag) == np.float32(oag)
            if ring is not None:
                assert_ring_matches(ring, oring)
            if with_db:
                for e, ref in enumerate(R.grouped_db(f32(G)[:used].astype(np.float64), off)):
                    if ref is None or off[e] == off[e + 1]:
                        assert not db[e].any()
                    else:
                        check_gemm(bf16_bits(db[e]), ref, f"db {e}")


def test_gradients_of_gradients_are_refused():
    from scaled_quantize_fp8_amd.autograd import Fp8GroupedLinear
    m = Fp8GroupedLinear(2, 32, 32, device=DEV)
    x = bf16((8, 32), 1.0, 1).to(DEV).requires_grad_(True)
    v = bf16((8, 32), 1.0, 2).to(DEV).requires_grad_(True)
    g, = torch.autograd.grad(m(x, offsets_dev([0, 4, 8])), x, v, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiate twice"):
        g.sum().backward()


def test_backward_with_different_weight_and_input_formats():
    """X8 in e4m3 beside W8 in e5m2 (the gradients' products then run as two
    launches)."""
    N, K = 96, 144
    T, off, E, x8, w8, sx, sw = _operands("edges", N, K, O.E4M3, O.E5M2)
    g8, sg = random_codes((T, N), 5, O.E5M2), np.float32(3.0)
    dx, dw, db = _filled(T, K), _filled(E, N, K), _filled(E, N)
    F.fp8_grouped_linear_bwd(F.Quantized(to_dev(g8), O.E5M2, scalar_dev(sg)), O.E5M2,
                             offsets_dev(off), F.Quantized(to_dev(x8), O.E4M3, scalar_dev(sx)),
                             F.Quantized(to_dev(w8), O.E5M2, to_dev(sw)), dx, dw, db)
    check_groups(dx, R.grouped_dx(g8, O.E5M2, w8, O.E5M2, sg, sw, off), off, "dx")
    dbs = R.grouped_db(O.dequantized(g8, O.E5M2, sg), off)
    for e, ref in enumerate(R.grouped_dw(g8, O.E5M2, x8, O.E4M3, sg, sx, off)):
        if ref is not None:
            check_gemm(bf16_bits(dw[e]), ref, f"dw {e}")
            check_gemm(bf16_bits(db[e]), dbs[e], f"db {e}")
