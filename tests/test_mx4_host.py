"""CPU checks of the 4-bit floating point entry points: the C ABI's refusals
(each returns before anything is enqueued) and the binding's."""

import ctypes

import pytest
import torch

import scaled_quantize_fp8_amd as F

P = ctypes.c_void_p(0x100000)  # a non-null "device" address never dereferenced
ODD = ctypes.c_void_p(0x100002)
Z = None
BF, E4, MX = F.FP8_DT_BF16, F.FP8_DT_E4M3, F.FP8_DT_MX4


@pytest.fixture(scope="module")
def lib():
    return F.lib()


def _lin(lib, M=4, N=16, K=64, x=P, dt=BF, xs=Z, w=P, ws=P, bias=Z, out=BF, y=P, x4=P, sx=P):
    return lib.fp8_mx4_linear_fwd(M, N, K, x, dt, xs, w, ws, bias, out, y, x4, sx, None)


def _glin(lib, M=4, N=16, K=64, x=P, dt=BF, xs=Z, w=P, ws=P, bias=Z, out=BF, y=P, x4=P, sx=P, E=2,
          off=P):
    return lib.fp8_mx4_grouped_linear_fwd(M, E, N, K, off, x, dt, xs, w, ws, bias, out, y, x4, sx,
                                          None)


@pytest.mark.parametrize("call", [_lin, _glin])
def test_linear_refusals(lib, call):
    for kw in (dict(M=-1), dict(N=-1), dict(K=-1), dict(K=1 << 24), dict(M=1 << 62),
               dict(M=1 << 31), dict(N=1 << 29, K=128), dict(M=1 << 25, K=128 * 16),
               dict(M=1 << 28, N=1 << 28, K=32)):
        assert call(lib, **kw) == F.FP8_ERR_SHAPE, kw
    for kw in (dict(out=F.FP8_DT_F32), dict(out=MX), dict(dt=E4), dict(dt=F.FP8_DT_I8), dict(dt=9)):
        assert call(lib, **kw) == F.FP8_ERR_DTYPE, kw
    for kw in (dict(x=Z), dict(x4=Z), dict(sx=Z), dict(dt=MX), dict(dt=MX, x=Z, xs=P), dict(w=Z),
               dict(ws=Z), dict(y=Z)):
        assert call(lib, **kw) == F.FP8_ERR_NULL, kw
    for kw in (dict(x4=ODD), dict(sx=ODD), dict(w=ODD), dict(ws=ODD), dict(dt=MX, xs=P, x=ODD),
               dict(dt=MX, xs=ODD)):
        assert call(lib, **kw) == F.FP8_ERR_SHAPE, kw
    assert _glin(lib, off=Z) == F.FP8_ERR_NULL and _glin(lib, E=0) == F.FP8_ERR_SHAPE


def test_quantize_refusals(lib):
    q = lib.fp8_mx4_quantize
    assert q(P, BF, 1, -1, 4, P, P, None) == F.FP8_ERR_SHAPE
    assert q(P, BF, 65536, 1, 4, P, P, None) == F.FP8_ERR_SHAPE
    assert q(P, BF, -1, 1, 4, P, P, None) == F.FP8_ERR_SHAPE
    assert q(P, BF, 1, 1, 1 << 24, P, P, None) == F.FP8_ERR_SHAPE
    assert q(P, E4, 1, 4, 4, P, P, None) == F.FP8_ERR_DTYPE
    for a in ((Z, P, P), (P, Z, P), (P, P, Z)):
        assert q(a[0], BF, 1, 4, 4, a[1], a[2], None) == F.FP8_ERR_NULL
    assert q(P, BF, 1, 4, 4, ODD, P, None) == F.FP8_ERR_SHAPE
    assert q(P, BF, 1, 4, 4, P, ODD, None) == F.FP8_ERR_SHAPE
    assert q(Z, BF, 0, 4, 4, Z, Z, None) == F.FP8_OK
    d = lib.fp8_mx4_dequantize
    assert d(P, P, 1, 4, -4, P, BF, None) == F.FP8_ERR_SHAPE
    assert d(P, P, 1, 4, 4, P, MX, None) == F.FP8_ERR_DTYPE
    for a in ((Z, P, P), (P, Z, P), (P, P, Z)):
        assert d(a[0], a[1], 1, 4, 4, a[2], BF, None) == F.FP8_ERR_NULL
    assert d(ODD, P, 1, 4, 4, P, BF, None) == F.FP8_ERR_SHAPE


def test_sizes():
    assert F.fp8_mx4_code_bytes(3, 33) == 3 * 32 and F.fp8_mx4_scale_bytes(3, 129) == 3 * 2 * 4
    assert F.fp8_mx4_code_bytes(-1, 33) == 0 and F.fp8_mx4_scale_bytes(4, 1 << 24) == 0
    q = F.QuantizedMx4.empty(2, 5, 200, device="cpu")
    assert q.codes.shape == (2, 5, 112) and q.scale.shape == (2, 2, 5, 4) and q.cols == 200
    assert q.codes.numel() == 2 * F.fp8_mx4_code_bytes(5, 200)
    assert q.scale.numel() == 2 * F.fp8_mx4_scale_bytes(5, 200)


def _t(*shape, dt=torch.bfloat16):
    return torch.zeros(*shape, dtype=dt)


_E = lambda *s: F.QuantizedMx4.empty(*s, device="cpu")


@pytest.mark.parametrize("call", [
    lambda: F.fp8_mx4_quantize(_t(64), _E(1, 64).codes, _E(1, 64).scale),
    lambda: F.fp8_mx4_quantize(_t(4, 64), _E(4, 96).codes, _E(4, 64).scale),
    lambda: F.fp8_mx4_quantize(_t(4, 64), _E(4, 64).codes, _E(4, 64).scale),  # not on the GPU
    lambda: F.fp8_mx4_dequantize(_E(4, 64), _t(4, 63)),
    lambda: F.fp8_mx4_linear_fwd(_t(4, 64), _E(16, 96), None, _t(4, 16), _E(4, 64).codes, _E(4, 64).scale),
    lambda: F.fp8_mx4_linear_fwd(_E(4, 96), _E(16, 64), None, _t(4, 16)),
    lambda: F.fp8_mx4_linear_fwd(_E(4, 64), _E(16, 64), None, _t(4, 15)),
    lambda: F.fp8_mx4_linear_fwd(_t(4, 64).T.contiguous().T, _E(16, 64), None, _t(4, 16)),
    lambda: F.fp8_mx4_grouped_linear_fwd(_E(4, 64), _E(16, 64), None, _t(3, dt=torch.int32), _t(4, 16)),
])
def test_binding_refuses_values(call):
    with pytest.raises(ValueError):
        call()


@pytest.mark.parametrize("call", [
    lambda: F.fp8_mx4_quantize(_t(4, 64, dt=torch.int32), _E(4, 64).codes, _E(4, 64).scale),
    lambda: F.fp8_mx4_dequantize(_t(4, 64), _t(4, 64)),
    lambda: F.fp8_mx4_linear_fwd(_E(4, 64), _t(16, 64), None, _t(4, 16)),
    lambda: F.fp8_mx4_grouped_linear_fwd(_E(4, 64), _t(2, 16, 64), None, _t(3), _t(4, 16)),
])
def test_binding_refuses_types(call):
    with pytest.raises(TypeError):
        call()
