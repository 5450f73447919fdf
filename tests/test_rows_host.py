"""CPU checks of the grouped and 8-bit integer entry points: the C ABI's
refusals (each returns before anything is enqueued) and the binding's."""

import ctypes

import pytest
import torch

import scaled_quantize_fp8_amd as F
from scaled_quantize_fp8_amd.int8 import Int8Linear

P = ctypes.c_void_p(0x100000)  # a non-null "device" address never dereferenced
Z = None
BF, E4, E5 = F.FP8_DT_BF16, F.FP8_DT_E4M3, F.FP8_DT_E5M2


@pytest.fixture(scope="module")
def lib():
    return F.lib()


def _op(dt, data=P, scale=P):
    return F._Operand(data, dt, scale)


def _fwd(lib, T=8, E=2, N=16, K=16, off=P, x=_op(E4), w=_op(E4), ns=1, bias=Z, fmt=F.FP8_E4M3,
         rx=Z, rw=Z, y=P, x8=P, w8=P, sx=P, sw=P, ax=P, aw=P):
    return lib.fp8_grouped_linear_fwd(T, E, N, K, off, x, w, ns, bias, fmt, rx, rw, y, x8, w8, sx,
                                      sw, ax, aw, None)


def _bwd(lib, T=8, E=2, N=16, K=16, off=P, g=_op(E5), fmt=F.FP8_E5M2, rg=Z, x8=_op(E4),
         w8=_op(E4), ns=1, dx=P, dw=P, db=P, ws=P, g8=P, sg=P, ag=P):
    return lib.fp8_grouped_linear_bwd(T, E, N, K, off, g, fmt, rg, x8, w8, ns, dx, dw, db, ws, g8,
                                      sg, ag, None)


@pytest.mark.parametrize("call", [_fwd, _bwd])
def test_grouped_sizes(lib, call):
    for kw in (dict(T=-1), dict(T=1 << 31), dict(E=0), dict(E=-3), dict(E=65536), dict(N=-1),
               dict(K=-1), dict(N=1 << 31), dict(T=(1 << 31) - 1, N=1 << 20), dict(T=1 << 28, N=1 << 18),
               dict(N=1 << 30, K=1 << 30, E=65535)):
        assert call(lib, **kw) == F.FP8_ERR_SHAPE, kw
    assert call(lib, off=Z) == F.FP8_ERR_NULL


@pytest.mark.parametrize("call", [_fwd, _bwd])
def test_grouped_row_numbers_end_a_tile_below_32_bits(lib, call):
    """T so large that the rows of a last tile, or of loads in flight behind
    it, would pass 2^31 is refused whatever the tile numbers are."""
    for T in ((1 << 31) - 17, (1 << 31) - 256, (1 << 31) - 1024):
        assert call(lib, T=T, E=1, N=1, K=1) == F.FP8_ERR_SHAPE, T


def test_grouped_fwd_refusals(lib):
    assert _fwd(lib, fmt=7) == F.FP8_ERR_DTYPE
    assert _fwd(lib, x=_op(E5)) == F.FP8_ERR_DTYPE
    assert _fwd(lib, w=_op(E5)) == F.FP8_ERR_DTYPE
    assert _fwd(lib, x=_op(F.FP8_DT_I8)) == F.FP8_ERR_DTYPE
    assert _fwd(lib, x=_op(E4, data=Z)) == F.FP8_ERR_NULL
    assert _fwd(lib, x=_op(E4, scale=Z)) == F.FP8_ERR_NULL
    assert _fwd(lib, w=_op(E4, scale=Z)) == F.FP8_ERR_NULL
    assert _fwd(lib, ns=3) == F.FP8_ERR_SHAPE and _fwd(lib, ns=0) == F.FP8_ERR_SHAPE
    assert _fwd(lib, y=Z) == F.FP8_ERR_NULL
    assert _fwd(lib, x=_op(BF), x8=Z) == F.FP8_ERR_NULL
    assert _fwd(lib, x=_op(BF), sx=Z) == F.FP8_ERR_NULL
    assert _fwd(lib, x=_op(BF), ax=Z) == F.FP8_ERR_NULL       # dynamic needs amax
    assert _fwd(lib, w=_op(BF), w8=Z) == F.FP8_ERR_NULL
    ring = F._Ring(P, 16, 1)
    assert _fwd(lib, x=_op(BF), w=_op(BF), rx=ctypes.byref(ring), sx=P) == F.FP8_ERR_RING
    r = ctypes.pointer(F._Ring(ctypes.c_void_p(0x500000), 16, 1))
    assert _fwd(lib, x=_op(BF), w=_op(BF), rx=r, rw=r) == F.FP8_ERR_RING


def test_grouped_bwd_refusals(lib):
    assert _bwd(lib, fmt=9) == F.FP8_ERR_DTYPE
    assert _bwd(lib, g=_op(E4)) == F.FP8_ERR_DTYPE
    assert _bwd(lib, g=_op(E5, data=Z)) == F.FP8_ERR_NULL
    assert _bwd(lib, g=_op(E5, scale=Z)) == F.FP8_ERR_NULL
    assert _bwd(lib, g=_op(BF), g8=Z) == F.FP8_ERR_NULL
    assert _bwd(lib, x8=_op(BF)) == F.FP8_ERR_DTYPE and _bwd(lib, w8=_op(BF)) == F.FP8_ERR_DTYPE
    assert _bwd(lib, x8=_op(E4, data=Z)) == F.FP8_ERR_NULL
    assert _bwd(lib, w8=_op(E4, scale=Z)) == F.FP8_ERR_NULL
    assert _bwd(lib, ns=5) == F.FP8_ERR_SHAPE
    assert _bwd(lib, g=_op(BF), ws=Z) == F.FP8_ERR_NULL
    ring = F._Ring(P, 0, 1)
    assert _bwd(lib, g=_op(BF), rg=ctypes.byref(ring)) == F.FP8_ERR_RING


def test_db_workspace():
    assert F.fp8_grouped_db_workspace_bytes(0, 4, 10) == 0
    assert F.fp8_grouped_db_workspace_bytes(1, 4, 10) == 40
    assert F.fp8_grouped_db_workspace_bytes(64, 1, 10) == 4 * 10 * 2
    # 64 rows in 2 groups: at most 3 chunks of 32
    assert F.fp8_grouped_db_workspace_bytes(64, 2, 10) == 4 * 10 * 3
    assert F.fp8_grouped_db_workspace_bytes(-1, 2, 10) == 0
    for T in range(1, 70):  # enough for every split into two groups
        most = max((a + 31) // 32 + (T - a + 31) // 32 for a in range(T + 1))
        assert F.fp8_grouped_db_workspace_bytes(T, 2, 1) >= 4 * most


I8 = F.FP8_DT_I8


def _lin(lib, M=4, N=16, K=16, x=_op(BF), w=_op(I8), bias=Z, out=BF, y=P, x8=P, sx=P):
    return lib.fp8_i8_linear_fwd(M, N, K, x, w, bias, out, y, x8, sx, None)


def _glin(lib, M=4, N=16, K=16, x=_op(BF), w=_op(I8), bias=Z, out=BF, y=P, x8=P, sx=P, E=2, off=P):
    return lib.fp8_i8_grouped_linear_fwd(M, E, N, K, off, x, w, bias, out, y, x8, sx, None)


@pytest.mark.parametrize("call", [_lin, _glin])
def test_i8_refusals(lib, call):
    for kw in (dict(M=-1), dict(N=-1), dict(K=-1), dict(K=131072), dict(M=1 << 62)):
        assert call(lib, **kw) == F.FP8_ERR_SHAPE, kw
    for kw in (dict(out=F.FP8_DT_F32), dict(out=E4), dict(w=_op(E4)), dict(w=_op(BF)),
               dict(x=_op(E4)), dict(x=_op(9))):
        assert call(lib, **kw) == F.FP8_ERR_DTYPE, kw
    for kw in (dict(x=_op(BF, data=Z)), dict(x8=Z), dict(sx=Z), dict(x=_op(I8, data=Z)),
               dict(x=_op(I8, scale=Z)), dict(w=_op(I8, data=Z)), dict(w=_op(I8, scale=Z)),
               dict(y=Z)):
        assert call(lib, **kw) == F.FP8_ERR_NULL, kw
    assert _glin(lib, off=Z) == F.FP8_ERR_NULL
    assert _glin(lib, E=0) == F.FP8_ERR_SHAPE


def test_i8_quantize_refusals(lib):
    q = lib.fp8_i8_quantize_rows
    assert q(P, BF, -1, 4, P, P, None) == F.FP8_ERR_SHAPE
    assert q(P, BF, 1 << 40, 1 << 40, P, P, None) == F.FP8_ERR_SHAPE
    assert q(P, E4, 4, 4, P, P, None) == F.FP8_ERR_DTYPE
    assert q(Z, BF, 4, 4, P, P, None) == F.FP8_ERR_NULL
    assert q(P, BF, 4, 4, Z, P, None) == F.FP8_ERR_NULL
    assert q(P, BF, 4, 4, P, Z, None) == F.FP8_ERR_NULL


# ---------------------------------------------------------------- binding

def _t(*shape, dt=torch.bfloat16):
    return torch.zeros(*shape, dtype=dt)


def _q(*shape, scales=1):
    return F.Quantized(_t(*shape, dt=torch.uint8), F.FP8_E4M3, torch.ones(scales))


OFF = torch.tensor([0, 3, 8], dtype=torch.int32)


def test_binding_host_tensors_raise():
    with pytest.raises(ValueError, match="GPU tensor"):
        F.fp8_grouped_linear_fwd(_q(8, 16), _q(2, 32, 16), None, OFF, F.FP8_E4M3, _t(8, 32))
    with pytest.raises(ValueError, match="GPU tensor"):
        F.fp8_i8_quantize_rows(_t(8, 16), _t(8, 16, dt=torch.int8), torch.ones(8))


@pytest.mark.parametrize("kw,err,match", [
    (dict(x=_q(16, 8)), ValueError, "shape"),                      # K differs
    (dict(x=F.Quantized(_t(16, 8, dt=torch.uint8).mT, 0, torch.ones(1))), ValueError, "contig"),
    (dict(w=_q(32, 16)), ValueError, "3-D"),
    (dict(x=_q(8, 16, scales=2)), ValueError, "scales"),
    (dict(w=_q(2, 32, 16, scales=3)), ValueError, "scales"),
    (dict(y=_t(8, 32, dt=torch.float16)), TypeError, "dtype"),
    (dict(y=_t(8, 31)), ValueError, "shape"),
    (dict(offsets=OFF.long()), TypeError, "dtype"),
    (dict(offsets=OFF[:2]), ValueError, "shape"),
    (dict(bias=_t(32)), ValueError, "shape"),
    (dict(bias=_t(2, 32, dt=torch.float32)), TypeError, "dtype"),
    (dict(x=None), TypeError, "Tensor|expected"),
])
def test_binding_grouped_forward_refuses(kw, err, match, monkeypatch):
    # host tensors stand for GPU ones: only the structural checks are under test
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))
    args = dict(x=_q(8, 16), w=_q(2, 32, 16), bias=None, offsets=OFF, fmt=F.FP8_E4M3, y=_t(8, 32))
    args.update(kw)
    with pytest.raises((err, ValueError), match=match):
        F.fp8_grouped_linear_fwd(**args)


@pytest.mark.parametrize("kw,match", [
    (dict(dx=_t(8, 15)), "shape"), (dict(dw=_t(2, 32, 15)), "shape"),
    (dict(db=_t(32)), "shape"), (dict(x8=None), "Quantized"), (dict(w8=_t(2, 32, 16)), "Quantized"),
    (dict(db_ws=_t(1)), "needed"), (dict(offsets=OFF[:1]), "offsets"),
    (dict(g8_out=_t(8, 32)), "dtype"),
])
def test_binding_grouped_backward_refuses(kw, match, monkeypatch):
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))
    args = dict(g=_t(8, 32), fmt_g=F.FP8_E5M2, offsets=OFF, x8=_q(8, 16), w8=_q(2, 32, 16),
                dx=_t(8, 16), dw=_t(2, 32, 16), db=_t(2, 32), db_ws=_t(4096))
    args.update(kw)
    with pytest.raises((ValueError, TypeError), match=match):
        F.fp8_grouped_linear_bwd(**args)


def _w8(*shape, scales=None):
    return F.QuantizedRows(_t(*shape, dt=torch.int8), torch.ones(shape[:-1] if scales is None
                                                                 else scales))


@pytest.mark.parametrize("kw,match", [
    (dict(x=_t(8, 15)), "shape"), (dict(w=_t(32, 16, dt=torch.int8)), "QuantizedRows"),
    (dict(w=_w8(32, 16, scales=1)), "shape"), (dict(y=_t(8, 32, dt=torch.float32)), "dtype"),
    (dict(bias=_t(32, dt=torch.float16)), "dtype"), (dict(bias=_t(31)), "shape"),
    (dict(x8_out=None), "x8_out"), (dict(sx_out=torch.ones(7)), "at least"),
    (dict(x8_out=_t(8, 16)), "dtype"), (dict(x=_t(16, 8).mT), "contiguous"),
    (dict(x=_w8(8, 16, scales=(8, 1))), "shape"),
])
def test_binding_i8_refuses(kw, match, monkeypatch):
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))
    args = dict(x=_t(8, 16), w=_w8(32, 16), bias=None, y=_t(8, 32),
                x8_out=_t(8, 16, dt=torch.int8), sx_out=torch.ones(8))
    args.update(kw)
    with pytest.raises((ValueError, TypeError), match=match):
        F.fp8_i8_linear_fwd(**args)


def test_int8_module_refuses_gradients():
    m = Int8Linear.__new__(Int8Linear)
    torch.nn.Module.__init__(m)
    with pytest.raises(RuntimeError, match="no gradient"):
        m.forward(torch.zeros(2, 4, requires_grad=True))


# ---------------------------------------------------------------- launch sizes

MANY = dict(T=65535, E=65535)  # one row per expert: every expert has its own tiles


def test_products_of_too_many_tiles_are_refused(lib):
    """A grid takes fewer than 2^32 threads: sizes whose general tiles (256
    threads for 128x128) pass that are refused before anything is enqueued."""
    assert _fwd(lib, **MANY, N=32896) == F.FP8_ERR_SHAPE        # 65535 x 257 tiles
    assert _fwd(lib, **MANY, N=32896, x=_op(BF), w=_op(BF)) == F.FP8_ERR_SHAPE
    assert _glin(lib, M=65535, E=65535, N=32896) == F.FP8_ERR_SHAPE
    assert _lin(lib, M=1, N=1 << 31, K=1) == F.FP8_ERR_SHAPE    # 2^24 tiles
    assert _lin(lib, M=(1 << 31) - 128, N=1, K=1) == F.FP8_ERR_SHAPE


def test_gradients_of_too_many_tiles_are_refused(lib):
    alone = dict(dx=Z, dw=Z, db=Z)
    assert _bwd(lib, **MANY, N=16, K=32896, **{**alone, "dx": P}) == F.FP8_ERR_SHAPE
    assert _bwd(lib, T=8, E=65535, N=2048, K=2048, **{**alone, "dw": P}) == F.FP8_ERR_SHAPE
    # db: 64 columns a block from the chunk sums, 256 from codes
    assert _bwd(lib, T=8, E=65535, N=16448, K=16, g=_op(BF), **{**alone, "db": P}) == F.FP8_ERR_SHAPE
    assert _bwd(lib, T=8, E=65535, N=65792, K=16, **{**alone, "db": P}) == F.FP8_ERR_SHAPE
    # the quantize's chunks of 32 rows by 256 columns
    assert _bwd(lib, T=1 << 29, E=1, N=8, K=16, g=_op(BF), **{**alone, "db": P}) == F.FP8_ERR_SHAPE
