"""CPU checks of the routing and exchange entry points: the C ABI's refusals
(each returns before anything is enqueued) and the binding's."""

import ctypes

import pytest
import torch

import scaled_quantize_fp8_amd as F

P = ctypes.c_void_p(0x100000)  # a non-null "device" address never dereferenced
Z = None
BF, E4 = F.FP8_DT_BF16, F.FP8_DT_E4M3


@pytest.fixture(scope="module")
def lib():
    return F.lib()


def _fwd(lib, T=8, E=8, k=2, z=P, dt=BF, b=Z, score=0, groups=1, kept=1, top=1, renorm=1, idx=P,
         w=P, off=P, pos=P, ws=P):
    return lib.fp8_route_fwd(T, E, k, z, dt, b, score, groups, kept, top, renorm, 1.0, idx, w, off,
                             pos, ws, None)


def _bwd(lib, T=8, E=8, k=2, z=P, dt=BF, score=0, idx=P, dw=P, dz=P):
    return lib.fp8_route_bwd(T, E, k, z, dt, score, 1, 1.0, idx, dw, dz, None)


def _plan(lib, T=8, E=8, k=2, idx=P, off=P, pos=P, ws=P):
    return lib.fp8_route_plan(T, E, k, idx, off, pos, ws, None)


@pytest.mark.parametrize("call", [_fwd, _bwd, _plan])
def test_sizes(lib, call):
    for kw in (dict(T=-1), dict(E=0), dict(E=1025), dict(k=0), dict(k=65, E=100),
               dict(T=(1 << 29) + 1), dict(T=1 << 62)):
        assert call(lib, **kw) == F.FP8_ERR_SHAPE, kw


def test_route_refusals(lib):
    for kw in (dict(k=9), dict(groups=3), dict(groups=0), dict(groups=4, kept=5),
               dict(groups=4, kept=0), dict(groups=8, kept=1), dict(top=3), dict(top=0)):
        assert _fwd(lib, **kw) == F.FP8_ERR_SHAPE, kw
    for kw in (dict(dt=E4), dict(dt=9), dict(score=2), dict(score=-1)):
        assert _fwd(lib, **kw) == F.FP8_ERR_DTYPE, kw
        assert _bwd(lib, **kw) == F.FP8_ERR_DTYPE, kw
    for kw in (dict(z=Z), dict(idx=Z), dict(w=Z), dict(off=Z), dict(pos=Z), dict(T=20000, ws=Z)):
        assert _fwd(lib, **kw) == F.FP8_ERR_NULL, kw
    for kw in (dict(z=Z), dict(idx=Z), dict(dw=Z), dict(dz=Z)):
        assert _bwd(lib, **kw) == F.FP8_ERR_NULL, kw
    assert _bwd(lib, k=9) == F.FP8_ERR_SHAPE
    for kw in (dict(idx=Z), dict(off=Z), dict(pos=Z), dict(T=20000, ws=Z)):
        assert _plan(lib, **kw) == F.FP8_ERR_NULL, kw
    assert _plan(lib, T=20000, ws=ctypes.c_void_p(0x100002)) == F.FP8_ERR_SHAPE


def test_workspace():
    w = F.fp8_route_workspace_bytes
    assert w(0, 8, 2) == 0 and w(16384, 8, 2) == 0 and w(16385, 8, 2) == 17 * 8 * 4
    assert w(-1, 8, 2) == 0 and w(10000, 2000, 2) == 0
    for T in (1 << 10, 1 << 17, 1 << 20, 1 << 24):  # at most 512 chunks' counts
        assert w(T, 256, 8) <= 512 * 256 * 4


def test_exchange_refusals(lib):
    g = lambda T=8, k=2, row=64, R=16, x=P, pos=P, out=P: lib.fp8_route_gather(
        T, k, row, R, x, pos, out, None)
    c = lambda T=8, k=2, D=64, R=16, y=P, dt=BF, pos=P, w=P, out=P: lib.fp8_route_combine(
        T, k, D, R, y, dt, pos, w, out, None)
    b = lambda T=8, k=2, D=64, R=16, do=P, y=P, dt=BF, pos=P, w=P, dy=P, dw=P: \
        lib.fp8_route_combine_bwd(T, k, D, R, do, y, dt, pos, w, dy, dw, None)
    for call in (g, c, b):
        for kw in (dict(T=-1), dict(k=0), dict(k=65), dict(R=-1), dict(R=1 << 31),
                   dict(T=1 << 30)):
            assert call(**kw) == F.FP8_ERR_SHAPE, kw
        assert call(pos=Z) == F.FP8_ERR_NULL
    assert g(row=-1) == F.FP8_ERR_SHAPE and g(row=1 << 24) == F.FP8_ERR_SHAPE
    assert g(x=Z) == F.FP8_ERR_NULL and g(out=Z) == F.FP8_ERR_NULL
    for call in (c, b):
        assert call(D=-1) == F.FP8_ERR_SHAPE and call(D=(1 << 22) + 1) == F.FP8_ERR_SHAPE
        assert call(dt=E4) == F.FP8_ERR_DTYPE
    assert c(y=Z) == F.FP8_ERR_NULL and c(out=Z) == F.FP8_ERR_NULL
    assert b(do=Z) == F.FP8_ERR_NULL and b(w=Z) == F.FP8_ERR_NULL and b(y=Z) == F.FP8_ERR_NULL
    # nothing to do: fine before any pointer is looked at
    assert g(T=0, x=Z, pos=Z, out=Z) == F.FP8_OK and c(T=0, y=Z, pos=Z, out=Z) == F.FP8_OK


# ---------------------------------------------------------------- binding

def _t(*shape, dt=torch.float32):
    return torch.zeros(*shape, dtype=dt)


I = torch.int32


@pytest.mark.parametrize("call", [
    lambda: F.fp8_route_fwd(_t(8), _t(8, 2, dt=I), _t(8, 2)),
    lambda: F.fp8_route_fwd(_t(8, 4), _t(8, 2, dt=I), _t(8, 3)),
    lambda: F.fp8_route_fwd(_t(8, 4), _t(7, 2, dt=I), _t(8, 2)),
    lambda: F.fp8_route_fwd(_t(8, 4).T.contiguous().T, _t(8, 2, dt=I), _t(8, 2)),
    lambda: F.fp8_route_fwd(_t(8, 4), _t(8, 2, dt=I), _t(8, 2)),       # not on the GPU
    lambda: F.fp8_route_bwd(_t(8, 4), _t(8, 2, dt=I), _t(8, 2), _t(8, 5)),
    lambda: F.fp8_route_plan(_t(8, 2, dt=I), _t(2, 5, dt=I), _t(8, 2, dt=I)),
    lambda: F.fp8_route_gather(_t(8, 4), _t(7, 2, dt=I), _t(16, 4)),
    lambda: F.fp8_route_gather(_t(8, 4), _t(8, 2, dt=I), _t(16, 5)),
    lambda: F.fp8_route_combine(_t(16, 4), _t(8, 2, dt=I), _t(8, 1), _t(8, 4)),
    lambda: F.fp8_route_combine_bwd(_t(8, 4), _t(16, 5), _t(8, 2, dt=I), _t(8, 2), _t(16, 4)),
])
def test_binding_refuses_values(call):
    with pytest.raises(ValueError):
        call()


@pytest.mark.parametrize("call", [
    lambda: F.fp8_route_fwd(_t(8, 4, dt=torch.float64), _t(8, 2, dt=I), _t(8, 2)),
    lambda: F.fp8_route_fwd(None, _t(8, 2, dt=I), _t(8, 2)),
    lambda: F.fp8_route_gather(None, _t(8, 2, dt=I), _t(16, 4)),
])
def test_binding_refuses_types(call):
    with pytest.raises((TypeError, ValueError)):
        call()
