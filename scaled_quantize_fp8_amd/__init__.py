"""Python binding of libfp8linear.so: argument marshalling only.

Every function here has the name of the C entry point it calls and maps
torch tensors (device memory) to the pointers and sizes of the C ABI
declared in include/fp8linear.h.  No step of the computation runs in
Python; without the built library every call raises.

Conventions: fmt / dtype values are the C enums below; pre-quantized
operands are passed as ``Quantized(codes_uint8, fmt, scale_f32)``; rings are
``ScaleRing`` objects that own their device buffer and the C struct; 8-bit
integer operands are ``QuantizedRows(codes_int8, scales_f32)``.
"""

from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

from ._build import LIB_PATH

FP8_E4M3, FP8_E5M2 = 0, 1
FP8_DT_F32, FP8_DT_F16, FP8_DT_BF16, FP8_DT_E4M3, FP8_DT_E5M2, FP8_DT_I8 = 0, 1, 2, 3, 4, 5
FP8_DT_MX4 = 6
FP8_OK, FP8_ERR_NULL, FP8_ERR_SHAPE, FP8_ERR_DTYPE, FP8_ERR_RING, FP8_ERR_HIP = range(6)
FP8_K_CONTIG, FP8_K_STRIDED = 0, 1
FP8_QUANT_ROWS, FP8_QUANT_TRANSPOSED, FP8_QUANT_DUAL = 0, 1, 2
FP8_ROUTE_SOFTMAX, FP8_ROUTE_SIGMOID = 0, 1

_TORCH_DT = {torch.float32: FP8_DT_F32, torch.float16: FP8_DT_F16, torch.bfloat16: FP8_DT_BF16}
_FMT_DT = {FP8_E4M3: FP8_DT_E4M3, FP8_E5M2: FP8_DT_E5M2}

C_SYMBOLS = (
    "fp8_abi_version", "fp8_source_hash", "fp8_status_str", "fp8_ring_bytes", "fp8_ring_init", "fp8_quantize",
    "fp8_quantize_pair", "fp8_linear_fwd", "fp8_linear_bwd_dx", "fp8_db_workspace_bytes",
    "fp8_linear_bwd_dw", "fp8_gemm", "fp8_quantize_2d", "fp8_gemm_fp8out", "fp8_linear_bwd",
    "fp8_linear_bwd_dw_noalloc", "fp8_grouped_db_workspace_bytes", "fp8_grouped_linear_fwd",
    "fp8_grouped_linear_bwd", "fp8_i8_quantize_rows", "fp8_i8_linear_fwd",
    "fp8_i8_grouped_linear_fwd", "fp8_route_workspace_bytes", "fp8_route_fwd", "fp8_route_bwd",
    "fp8_route_plan", "fp8_route_gather", "fp8_route_combine", "fp8_route_combine_bwd",
    "fp8_mx4_code_bytes", "fp8_mx4_scale_bytes", "fp8_mx4_quantize", "fp8_mx4_dequantize",
    "fp8_mx4_linear_fwd", "fp8_mx4_grouped_linear_fwd",
)


class Fp8Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_str(status)} (status {status})")


class _Operand(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("scale", ctypes.c_void_p)]


class _Ring(ctypes.Structure):
    _fields_ = [("dev", ctypes.c_void_p), ("hist_len", ctypes.c_int32), ("seeded", ctypes.c_int32)]


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded HIP library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built (run __graft_entry__.build())")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        op, rp = _Operand, ctypes.POINTER(_Ring)
        L.fp8_abi_version.restype = ctypes.c_int
        L.fp8_source_hash.restype = ctypes.c_char_p
        L.fp8_source_hash.argtypes = []
        L.fp8_status_str.restype = ctypes.c_char_p
        L.fp8_status_str.argtypes = [ctypes.c_int]
        L.fp8_ring_bytes.restype = sz
        L.fp8_ring_bytes.argtypes = [i32]
        L.fp8_db_workspace_bytes.restype = sz
        L.fp8_db_workspace_bytes.argtypes = [i64, i64]
        L.fp8_ring_init.argtypes = [rp, vp, i32, vp]
        L.fp8_quantize.argtypes = [vp, i32, i64, i32, vp, rp, vp, vp, vp]
        L.fp8_quantize_pair.argtypes = [vp, i32, i64, vp, rp, vp, vp, vp, i32, i64, vp, rp, vp, vp,
                                        i32, vp]
        L.fp8_linear_fwd.argtypes = [i64, i64, i64, op, op, op, i32, rp, rp, vp, vp, vp, vp, vp, vp,
                                     vp, vp]
        L.fp8_linear_bwd_dx.argtypes = [i64, i64, i64, op, i32, rp, op, vp, vp, vp, vp, vp]
        L.fp8_linear_bwd_dw.argtypes = [i64, i64, i64, op, i32, rp, op, vp, vp, vp, vp, vp, vp, vp]
        L.fp8_linear_bwd_dw_noalloc.argtypes = [i64, i64, i64, op, i32, rp, op, vp, vp, vp, vp, vp,
                                                vp]
        L.fp8_linear_bwd.argtypes = [i64, i64, i64, op, i32, rp, op, op, vp, vp, vp, vp, vp, vp, vp,
                                     vp, vp]
        L.fp8_quantize_2d.argtypes = [vp, i32, i64, i64, i32, i32, vp, vp, rp, vp, vp, vp]
        L.fp8_gemm.argtypes = [i64, i64, i64, i64, op, i32, i64, i64, op, i32, i64, i64, op, vp,
                               i64, i64, vp]
        L.fp8_gemm_fp8out.argtypes = [i64, i64, i64, op, op, op, i32, rp, vp, vp, vp, vp]
        L.fp8_grouped_db_workspace_bytes.restype = sz
        L.fp8_grouped_db_workspace_bytes.argtypes = [i64, i32, i64]
        L.fp8_grouped_linear_fwd.argtypes = [i64, i32, i64, i64, vp, op, op, i32, vp, i32, rp, rp,
                                             vp, vp, vp, vp, vp, vp, vp, vp]
        L.fp8_grouped_linear_bwd.argtypes = [i64, i32, i64, i64, vp, op, i32, rp, op, op, i32, vp,
                                             vp, vp, vp, vp, vp, vp, vp]
        L.fp8_i8_quantize_rows.argtypes = [vp, i32, i64, i64, vp, vp, vp]
        L.fp8_i8_linear_fwd.argtypes = [i64, i64, i64, op, op, vp, i32, vp, vp, vp, vp]
        L.fp8_i8_grouped_linear_fwd.argtypes = [i64, i32, i64, i64, vp, op, op, vp, i32, vp, vp, vp,
                                                vp]
        f32 = ctypes.c_float
        L.fp8_route_workspace_bytes.restype = sz
        L.fp8_route_workspace_bytes.argtypes = [i64, i32, i32]
        L.fp8_route_fwd.argtypes = [i64, i32, i32, vp, i32, vp, i32, i32, i32, i32, i32, f32, vp, vp,
                                    vp, vp, vp, vp]
        L.fp8_route_bwd.argtypes = [i64, i32, i32, vp, i32, i32, i32, f32, vp, vp, vp, vp]
        L.fp8_route_plan.argtypes = [i64, i32, i32, vp, vp, vp, vp, vp]
        L.fp8_route_gather.argtypes = [i64, i32, i64, i64, vp, vp, vp, vp]
        L.fp8_route_combine.argtypes = [i64, i32, i64, i64, vp, i32, vp, vp, vp, vp]
        L.fp8_route_combine_bwd.argtypes = [i64, i32, i64, i64, vp, vp, i32, vp, vp, vp, vp, vp]
        L.fp8_mx4_code_bytes.restype = L.fp8_mx4_scale_bytes.restype = sz
        L.fp8_mx4_code_bytes.argtypes = L.fp8_mx4_scale_bytes.argtypes = [i64, i64]
        L.fp8_mx4_quantize.argtypes = [vp, i32, i64, i64, i64, vp, vp, vp]
        L.fp8_mx4_dequantize.argtypes = [vp, vp, i64, i64, i64, vp, i32, vp]
        L.fp8_mx4_linear_fwd.argtypes = [i64, i64, i64, vp, i32, vp, vp, vp, vp, i32, vp, vp, vp, vp]
        L.fp8_mx4_grouped_linear_fwd.argtypes = [i64, i32, i64, i64, vp, vp, i32, vp, vp, vp, vp,
                                                 i32, vp, vp, vp, vp]
        for name in ("fp8_route_fwd", "fp8_route_bwd", "fp8_route_plan", "fp8_route_gather",
                     "fp8_route_combine", "fp8_route_combine_bwd", "fp8_mx4_quantize",
                     "fp8_mx4_dequantize", "fp8_mx4_linear_fwd", "fp8_mx4_grouped_linear_fwd"):
            getattr(L, name).restype = ctypes.c_int
        for name in ("fp8_grouped_linear_fwd", "fp8_grouped_linear_bwd", "fp8_i8_quantize_rows",
                     "fp8_i8_linear_fwd", "fp8_i8_grouped_linear_fwd"):
            getattr(L, name).restype = ctypes.c_int
        for name in ("fp8_ring_init", "fp8_quantize", "fp8_quantize_pair", "fp8_quantize_2d",
                     "fp8_linear_fwd", "fp8_gemm", "fp8_linear_bwd_dx",
                     "fp8_linear_bwd_dw", "fp8_gemm_fp8out", "fp8_linear_bwd",
                     "fp8_linear_bwd_dw_noalloc"):
            getattr(L, name).restype = ctypes.c_int
        _lib = L
    return _lib


def status_str(status: int) -> str:
    return lib().fp8_status_str(status).decode()


def fp8_abi_version() -> int:
    return lib().fp8_abi_version()


def fp8_source_hash() -> str:
    return lib().fp8_source_hash().decode()


def fp8_ring_bytes(hist_len: int) -> int:
    return lib().fp8_ring_bytes(hist_len)


def fp8_db_workspace_bytes(M: int, N: int) -> int:
    return lib().fp8_db_workspace_bytes(M, N)


def fp8_grouped_db_workspace_bytes(T: int, E: int, N: int) -> int:
    return lib().fp8_grouped_db_workspace_bytes(T, E, N)


def fp8_mx4_code_bytes(rows: int, K: int) -> int:
    return lib().fp8_mx4_code_bytes(rows, K)


def fp8_mx4_scale_bytes(rows: int, K: int) -> int:
    return lib().fp8_mx4_scale_bytes(rows, K)


def fp8_route_workspace_bytes(T: int, E: int, k: int) -> int:
    return lib().fp8_route_workspace_bytes(T, E, k)


# ---------------------------------------------------------------- marshalling

def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _check(status: int, where: str) -> None:
    if status != FP8_OK:
        raise Fp8Error(status, where)


_HP = (torch.float32, torch.float16, torch.bfloat16)


def _need(t, what, dtypes=None, shape=None, numel=None, optional=True):
    """Validate a tensor argument before its pointer crosses the boundary:
    contiguous (the C ABI takes dense row-major buffers: a transposed or
    strided view would be read as the wrong elements), of an allowed dtype,
    of the expected shape or element count, on the GPU.  None passes when
    the argument is optional (the library decides whether it is needed)."""
    if t is None:
        if optional:
            return
        raise ValueError(f"{what} is required")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what}: expected a torch.Tensor, got {type(t).__name__}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: must be contiguous (shape {tuple(t.shape)}, "
                         f"strides {t.stride()}); pass .contiguous()")
    if dtypes is not None and t.dtype not in dtypes:
        raise TypeError(f"{what}: dtype {t.dtype} not in {[str(d) for d in dtypes]}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if numel is not None and t.numel() < numel:
        raise ValueError(f"{what}: {t.numel()} elements, at least {numel} needed")


def _on_gpu(**named):
    """Second phase of the checks, after every argument's structure: each
    tensor (or Quantized operand) given lives on the GPU."""
    for what, t in named.items():
        for name, x in ((what, t.codes), (what + ".scale", t.scale)) if isinstance(t, Quantized) \
                else ((what, t),):
            if isinstance(x, torch.Tensor) and x.device.type != "cuda":
                raise ValueError(f"{name}: must be a GPU tensor (got {x.device})")


def _need_scalar(t, what, optional=True):
    _need(t, what, (torch.float32,), numel=1, optional=optional)


def _need_operand(t, what, shape, hp_ok=True):
    """A high-precision tensor or a Quantized (uint8 codes + float32 scale)."""
    if isinstance(t, Quantized):
        _need(t.codes, f"{what}.codes", (torch.uint8,), shape=shape, optional=False)
        _need_scalar(t.scale, f"{what}.scale", optional=False)
        if t.fmt not in _FMT_DT:
            raise ValueError(f"{what}: unknown fp8 format {t.fmt}")
    elif hp_ok:
        _need(t, what, _HP, shape=shape, optional=False)
    else:
        raise TypeError(f"{what}: expected a Quantized operand")


def _dims2(t, what):
    d = t.codes if isinstance(t, Quantized) else t
    if not isinstance(d, torch.Tensor) or d.dim() != 2:
        raise ValueError(f"{what}: expected a 2-D matrix")
    return d.shape


@dataclass
class Quantized:
    """Pre-quantized operand: uint8 codes, format, device float32 scale [1]."""
    codes: torch.Tensor
    fmt: int
    scale: torch.Tensor


def _operand(t) -> _Operand:
    if t is None:
        return _Operand(None, FP8_DT_BF16, None)
    if isinstance(t, Quantized):
        return _Operand(_ptr(t.codes), _FMT_DT[t.fmt], _ptr(t.scale))
    return _Operand(_ptr(t), _TORCH_DT[t.dtype], None)


class ScaleRing:
    """Delayed-scaling ring: device buffer plus the C struct (seeded mirror)."""

    def __init__(self, hist_len: int, device="cuda", stream=None):
        nbytes = fp8_ring_bytes(hist_len)
        if nbytes == 0:
            raise Fp8Error(FP8_ERR_RING, "ScaleRing")
        self.buf = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.c = _Ring()
        _check(lib().fp8_ring_init(ctypes.byref(self.c), self.buf.data_ptr(), hist_len,
                                   _stream(stream)), "fp8_ring_init")

    @property
    def seeded(self) -> bool:
        return bool(self.c.seeded)

    def ref(self):
        return ctypes.byref(self.c)


def _ring(r):
    return None if r is None else r.ref()


# ---------------------------------------------------------------- entry points
# Each entry point has a *_args helper that turns tensors into the C argument
# tuple (marshalling), the call itself, and a bind_* variant that marshals
# once and returns a zero-argument callable (for launch-bound loops and graph
# capture: the pointers, sizes and stream are fixed at bind time).

def _vp(t):
    return ctypes.c_void_p(_ptr(t))


def _quantize_args(x, fmt, q, ring, scale_used, amax_out, stream):
    _need(x, "x", _HP, optional=False)
    _need(q, "q", (torch.uint8,), numel=x.numel(), optional=x.numel() == 0)
    _need_scalar(scale_used, "scale_used")
    _need_scalar(amax_out, "amax_out")
    _on_gpu(x=x, q=q, scale_used=scale_used, amax_out=amax_out)
    return (_vp(x), ctypes.c_int32(_TORCH_DT[x.dtype]), ctypes.c_int64(x.numel()),
            ctypes.c_int32(fmt), _vp(q), _ring(ring), _vp(scale_used), _vp(amax_out),
            ctypes.c_void_p(_stream(stream)))


def _quantize_pair_args(x0, q0, ring0, su0, am0, x1, q1, ring1, su1, am1, fmt, stream):
    for i, (x, q, su, am) in enumerate(((x0, q0, su0, am0), (x1, q1, su1, am1))):
        _need(x, f"x{i}", _HP, optional=False)
        _need(q, f"q{i}", (torch.uint8,), numel=x.numel(), optional=x.numel() == 0)
        _need_scalar(su, f"scale_used{i}")
        _need_scalar(am, f"amax_out{i}")
    _on_gpu(x0=x0, q0=q0, su0=su0, am0=am0, x1=x1, q1=q1, su1=su1, am1=am1)
    return (_vp(x0), ctypes.c_int32(_TORCH_DT[x0.dtype]), ctypes.c_int64(x0.numel()), _vp(q0),
            _ring(ring0), _vp(su0), _vp(am0), _vp(x1), ctypes.c_int32(_TORCH_DT[x1.dtype]),
            ctypes.c_int64(x1.numel()), _vp(q1), _ring(ring1), _vp(su1), _vp(am1),
            ctypes.c_int32(fmt), ctypes.c_void_p(_stream(stream)))


def _fwd_args(x, w, bias, fmt, y, ring_x, ring_w, x8_out, w8_out, sx_used, sw_used, amax_x,
              amax_w, stream):
    M, K = _dims2(x, "x")
    N = _dims2(w, "w")[0]
    _need_operand(x, "x", (M, K))
    _need_operand(w, "w", (N, K))
    if bias is not None:
        if isinstance(bias, Quantized):
            _need_operand(bias, "bias", (N,), hp_ok=False)
        else:
            _need(bias, "bias", (torch.bfloat16,), shape=(N,))
    _need(y, "y", (torch.bfloat16,), shape=(M, N), optional=M * N == 0)
    _need(x8_out, "x8_out", (torch.uint8,), shape=(M, K))
    _need(w8_out, "w8_out", (torch.uint8,), shape=(N, K))
    for t, n in ((sx_used, "sx_used"), (sw_used, "sw_used"), (amax_x, "amax_x"),
                 (amax_w, "amax_w")):
        _need_scalar(t, n)
    _on_gpu(x=x, w=w, bias=bias, y=y, x8_out=x8_out, w8_out=w8_out, sx_used=sx_used,
            sw_used=sw_used, amax_x=amax_x, amax_w=amax_w)
    return (ctypes.c_int64(M), ctypes.c_int64(N), ctypes.c_int64(K), _operand(x), _operand(w),
            _operand(bias), ctypes.c_int32(fmt), _ring(ring_x), _ring(ring_w), _vp(y), _vp(x8_out),
            _vp(w8_out), _vp(sx_used), _vp(sw_used), _vp(amax_x), _vp(amax_w),
            ctypes.c_void_p(_stream(stream)))


def _dx_args(g, fmt_g, w8, dx, ring_g, g8_out, sg_used, amax_g, stream):
    M, N = _dims2(g, "g")
    K = _dims2(w8, "w8")[1]
    _need_operand(g, "g", (M, N))
    _need_operand(w8, "w8", (N, K), hp_ok=False)
    _need(dx, "dx", (torch.bfloat16,), shape=(M, K), optional=M * K == 0)
    _need(g8_out, "g8_out", (torch.uint8,), shape=(M, N))
    _need_scalar(sg_used, "sg_used")
    _need_scalar(amax_g, "amax_g")
    _on_gpu(g=g, w8=w8, dx=dx, g8_out=g8_out, sg_used=sg_used, amax_g=amax_g)
    return (ctypes.c_int64(M), ctypes.c_int64(N), ctypes.c_int64(K), _operand(g),
            ctypes.c_int32(fmt_g), _ring(ring_g), _operand(w8), _vp(dx), _vp(g8_out),
            _vp(sg_used), _vp(amax_g), ctypes.c_void_p(_stream(stream)))


def _dw_args(g, fmt_g, x8, dw, db, db_ws, ring_g, g8_out, sg_used, amax_g, stream):
    M, N = _dims2(g, "g")
    K = _dims2(x8, "x8")[1]
    _need_operand(g, "g", (M, N))
    _need_operand(x8, "x8", (M, K), hp_ok=False)
    _need(dw, "dw", (torch.bfloat16,), shape=(N, K), optional=N * K == 0)
    _need(db, "db", (torch.bfloat16,), shape=(N,))
    _need(db_ws, "db_ws", (torch.float32,), numel=fp8_db_workspace_bytes(M, N) // 4)
    _need(g8_out, "g8_out", (torch.uint8,), shape=(M, N))
    _need_scalar(sg_used, "sg_used")
    _need_scalar(amax_g, "amax_g")
    _on_gpu(g=g, x8=x8, dw=dw, db=db, db_ws=db_ws, g8_out=g8_out, sg_used=sg_used, amax_g=amax_g)
    return (ctypes.c_int64(M), ctypes.c_int64(N), ctypes.c_int64(K), _operand(g),
            ctypes.c_int32(fmt_g), _ring(ring_g), _operand(x8), _vp(dw), _vp(db), _vp(db_ws),
            _vp(g8_out), _vp(sg_used), _vp(amax_g), ctypes.c_void_p(_stream(stream)))


def _bind(name, args):
    fn = getattr(lib(), name)

    def call():
        st = fn(*args)
        if st != FP8_OK:
            raise Fp8Error(st, name)
    return call


def fp8_quantize(x, fmt, q, ring=None, scale_used=None, amax_out=None, stream=None):
    _check(lib().fp8_quantize(*_quantize_args(x, fmt, q, ring, scale_used, amax_out, stream)),
           "fp8_quantize")


def bind_fp8_quantize(x, fmt, q, ring=None, scale_used=None, amax_out=None, stream=None):
    return _bind("fp8_quantize", _quantize_args(x, fmt, q, ring, scale_used, amax_out, stream))


def _quantize_2d_args(x, fmt, layout, q, qt, ring, scale_used, amax_out, stream):
    _need(x, "x", _HP, optional=False)
    if x.dim() != 2:
        raise ValueError("x: expected a 2-D matrix")
    rows, cols = x.shape
    _need(q, "q", (torch.uint8,), shape=(rows, cols))
    _need(qt, "qt", (torch.uint8,), shape=(cols, rows))
    _need_scalar(scale_used, "scale_used")
    _need_scalar(amax_out, "amax_out")
    _on_gpu(x=x, q=q, qt=qt, scale_used=scale_used, amax_out=amax_out)
    return (_vp(x), ctypes.c_int32(_TORCH_DT[x.dtype]), ctypes.c_int64(rows), ctypes.c_int64(cols),
            ctypes.c_int32(fmt), ctypes.c_int32(layout), _vp(q), _vp(qt), _ring(ring),
            _vp(scale_used), _vp(amax_out), ctypes.c_void_p(_stream(stream)))


def fp8_quantize_2d(x, fmt, layout, q=None, qt=None, ring=None, scale_used=None, amax_out=None,
                    stream=None):
    """x [rows, cols] -> q [rows, cols] and/or qt [cols, rows] (layout:
    FP8_QUANT_ROWS / _TRANSPOSED / _DUAL)."""
    _check(lib().fp8_quantize_2d(*_quantize_2d_args(x, fmt, layout, q, qt, ring, scale_used,
                                                    amax_out, stream)), "fp8_quantize_2d")


def bind_fp8_quantize_2d(x, fmt, layout, q=None, qt=None, ring=None, scale_used=None,
                         amax_out=None, stream=None):
    return _bind("fp8_quantize_2d", _quantize_2d_args(x, fmt, layout, q, qt, ring, scale_used,
                                                      amax_out, stream))


def fp8_quantize_pair(x0, q0, ring0, su0, am0, x1, q1, ring1, su1, am1, fmt, stream=None):
    """Two quantizes (x0 -> q0 with ring0, x1 -> q1 with ring1) in one call."""
    _check(lib().fp8_quantize_pair(*_quantize_pair_args(x0, q0, ring0, su0, am0, x1, q1, ring1,
                                                        su1, am1, fmt, stream)),
           "fp8_quantize_pair")


def bind_fp8_quantize_pair(x0, q0, ring0, su0, am0, x1, q1, ring1, su1, am1, fmt, stream=None):
    return _bind("fp8_quantize_pair", _quantize_pair_args(x0, q0, ring0, su0, am0, x1, q1, ring1,
                                                          su1, am1, fmt, stream))


def fp8_linear_fwd(x, w, bias, fmt, y, ring_x=None, ring_w=None, x8_out=None, w8_out=None,
                   sx_used=None, sw_used=None, amax_x=None, amax_w=None, stream=None):
    """x: [M,K] tensor or Quantized; w: [N,K] tensor or Quantized; bias: None,
    a bf16 [N] tensor or Quantized (fp8 codes with bias_scale)."""
    _check(lib().fp8_linear_fwd(*_fwd_args(x, w, bias, fmt, y, ring_x, ring_w, x8_out, w8_out,
                                           sx_used, sw_used, amax_x, amax_w, stream)),
           "fp8_linear_fwd")


def bind_fp8_linear_fwd(x, w, bias, fmt, y, ring_x=None, ring_w=None, x8_out=None, w8_out=None,
                        sx_used=None, sw_used=None, amax_x=None, amax_w=None, stream=None):
    return _bind("fp8_linear_fwd", _fwd_args(x, w, bias, fmt, y, ring_x, ring_w, x8_out, w8_out,
                                             sx_used, sw_used, amax_x, amax_w, stream))


def fp8_linear_bwd_dx(g, fmt_g, w8, dx, ring_g=None, g8_out=None, sg_used=None, amax_g=None,
                      stream=None):
    _check(lib().fp8_linear_bwd_dx(*_dx_args(g, fmt_g, w8, dx, ring_g, g8_out, sg_used, amax_g,
                                             stream)), "fp8_linear_bwd_dx")


def bind_fp8_linear_bwd_dx(g, fmt_g, w8, dx, ring_g=None, g8_out=None, sg_used=None, amax_g=None,
                           stream=None):
    return _bind("fp8_linear_bwd_dx", _dx_args(g, fmt_g, w8, dx, ring_g, g8_out, sg_used, amax_g,
                                               stream))


def fp8_linear_bwd_dw(g, fmt_g, x8, dw, db=None, db_ws=None, ring_g=None, g8_out=None,
                      sg_used=None, amax_g=None, stream=None):
    _check(lib().fp8_linear_bwd_dw(*_dw_args(g, fmt_g, x8, dw, db, db_ws, ring_g, g8_out,
                                             sg_used, amax_g, stream)), "fp8_linear_bwd_dw")


def bind_fp8_linear_bwd_dw(g, fmt_g, x8, dw, db=None, db_ws=None, ring_g=None, g8_out=None,
                           sg_used=None, amax_g=None, stream=None):
    return _bind("fp8_linear_bwd_dw", _dw_args(g, fmt_g, x8, dw, db, db_ws, ring_g, g8_out,
                                               sg_used, amax_g, stream))


def _dw_noalloc_args(g, fmt_g, x8, dw, db, ring_g, g8_out, sg_used, amax_g, stream):
    args = _dw_args(g, fmt_g, x8, dw, db, None, ring_g, g8_out, sg_used, amax_g, stream)
    return args[:9] + args[10:]  # the same arguments without db_ws


def fp8_linear_bwd_dw_noalloc(g, fmt_g, x8, dw, db=None, ring_g=None, g8_out=None, sg_used=None,
                              amax_g=None, stream=None):
    """fp8_linear_bwd_dw without a workspace: the db partials live in the
    library's static per-GPU array (no allocation; calls that overlap on one
    GPU race on it)."""
    _check(lib().fp8_linear_bwd_dw_noalloc(*_dw_noalloc_args(g, fmt_g, x8, dw, db, ring_g, g8_out,
                                                             sg_used, amax_g, stream)),
           "fp8_linear_bwd_dw_noalloc")


def bind_fp8_linear_bwd_dw_noalloc(g, fmt_g, x8, dw, db=None, ring_g=None, g8_out=None,
                                   sg_used=None, amax_g=None, stream=None):
    return _bind("fp8_linear_bwd_dw_noalloc", _dw_noalloc_args(g, fmt_g, x8, dw, db, ring_g,
                                                               g8_out, sg_used, amax_g, stream))


def _bwd_args(g, fmt_g, x8, w8, dx, dw, db, db_ws, ring_g, g8_out, sg_used, amax_g, stream,
              stream_dw):
    M, N = _dims2(g, "g")
    K = _dims2(x8, "x8")[1]
    _need_operand(g, "g", (M, N))
    _need_operand(x8, "x8", (M, K), hp_ok=False)
    _need_operand(w8, "w8", (N, K), hp_ok=False)
    _need(dx, "dx", (torch.bfloat16,), shape=(M, K), optional=M * K == 0)
    _need(dw, "dw", (torch.bfloat16,), shape=(N, K), optional=N * K == 0)
    _need(db, "db", (torch.bfloat16,), shape=(N,))
    _need(db_ws, "db_ws", (torch.float32,), numel=fp8_db_workspace_bytes(M, N) // 4)
    _need(g8_out, "g8_out", (torch.uint8,), shape=(M, N))
    _need_scalar(sg_used, "sg_used")
    _need_scalar(amax_g, "amax_g")
    _on_gpu(g=g, x8=x8, w8=w8, dx=dx, dw=dw, db=db, db_ws=db_ws, g8_out=g8_out, sg_used=sg_used,
            amax_g=amax_g)
    st = _stream(stream)
    st_dw = st if stream_dw is None else stream_dw.cuda_stream
    return (ctypes.c_int64(M), ctypes.c_int64(N), ctypes.c_int64(K), _operand(g),
            ctypes.c_int32(fmt_g), _ring(ring_g), _operand(x8), _operand(w8), _vp(dx), _vp(dw),
            _vp(db), _vp(db_ws), _vp(g8_out), _vp(sg_used), _vp(amax_g), ctypes.c_void_p(st),
            ctypes.c_void_p(st_dw))


def fp8_linear_bwd(g, fmt_g, x8, w8, dx, dw, db=None, db_ws=None, ring_g=None, g8_out=None,
                   sg_used=None, amax_g=None, stream=None, stream_dw=None):
    """Both gradients from one quantize of g: dX on stream, dW (and db) on
    stream_dw after the quantize (stream_dw None: the same stream)."""
    _check(lib().fp8_linear_bwd(*_bwd_args(g, fmt_g, x8, w8, dx, dw, db, db_ws, ring_g, g8_out,
                                           sg_used, amax_g, stream, stream_dw)), "fp8_linear_bwd")


def bind_fp8_linear_bwd(g, fmt_g, x8, w8, dx, dw, db=None, db_ws=None, ring_g=None, g8_out=None,
                        sg_used=None, amax_g=None, stream=None, stream_dw=None):
    return _bind("fp8_linear_bwd", _bwd_args(g, fmt_g, x8, w8, dx, dw, db, db_ws, ring_g, g8_out,
                                             sg_used, amax_g, stream, stream_dw))


def _matrix_view(t, what):
    """(batch, rows, cols, batch_stride, layout, ld) of a 2-D or 3-D tensor
    whose last two dims are (rows, k): k-contiguous rows, or the transposed
    view of such rows (k strided).  A batch dim of size 1 or stride 0 is
    broadcast."""
    if t.dim() == 2:
        t3, bstride = t.unsqueeze(0), 0
    elif t.dim() == 3:
        t3, bstride = t, (0 if t.shape[0] == 1 else t.stride(0))
    else:
        raise ValueError(f"{what}: expected a 2-D or 3-D tensor")
    B, R, Kd = t3.shape
    if t3.stride(2) == 1 or Kd <= 1:
        return B, R, Kd, bstride, FP8_K_CONTIG, max(t3.stride(1), Kd, 1)
    if t3.stride(1) == 1 or R <= 1:
        return B, R, Kd, bstride, FP8_K_STRIDED, max(t3.stride(2), R, 1)
    raise ValueError(f"{what}: neither dim of the matrix is contiguous")


def _gemm_args(a, b, c, bias, stream):
    Ba, M, K, sa, la, lda = _matrix_view(a.codes, "a")
    Bb, N, Kb, sb, lb, ldb = _matrix_view(b.codes, "b")
    if K != Kb:
        raise ValueError("a and b disagree on K")
    batch = max(Ba, Bb)
    if Ba not in (1, batch) or Bb not in (1, batch):
        raise ValueError("batch sizes do not broadcast")
    c3 = c if c.dim() == 3 else c.unsqueeze(0)
    if tuple(c3.shape) != (batch, M, N) or c3.stride(2) != 1:
        raise ValueError("c must be [batch, M, N] (or [M, N]) with contiguous rows")
    return (ctypes.c_int64(batch), ctypes.c_int64(M), ctypes.c_int64(N), ctypes.c_int64(K),
            _operand(a), ctypes.c_int32(la), ctypes.c_int64(lda), ctypes.c_int64(sa),
            _operand(b), ctypes.c_int32(lb), ctypes.c_int64(ldb), ctypes.c_int64(sb),
            _operand(bias), _vp(c), ctypes.c_int64(max(c3.stride(1), N)),
            ctypes.c_int64(c3.stride(0) if batch > 1 else 0), ctypes.c_void_p(_stream(stream)))


def fp8_gemm(a, b, c, bias=None, stream=None):
    """c[z] = a[z] b[z]^T / (sa sb) (+ bias), bf16.  a: Quantized with codes
    [.., M, K]; b: Quantized with codes [.., N, K]; either may be a transposed
    view (.mT of a [.., K, M] buffer) and either may be 2-D or have batch 1
    (broadcast).  c: bf16 [.., M, N]."""
    _check(lib().fp8_gemm(*_gemm_args(a, b, c, bias, stream)), "fp8_gemm")


def bind_fp8_gemm(a, b, c, bias=None, stream=None):
    return _bind("fp8_gemm", _gemm_args(a, b, c, bias, stream))



def _gemm_fp8out_args(a, b, c8, fmt_out, ring_out, scale_used, amax_out, bias, stream):
    M, K = _dims2(a, "a")
    N = _dims2(b, "b")[0]
    _need_operand(a, "a", (M, K), hp_ok=False)
    _need_operand(b, "b", (N, K), hp_ok=False)
    _need(c8, "c8", (torch.uint8,), shape=(M, N), optional=False)
    _need_scalar(scale_used, "scale_used")
    _need_scalar(amax_out, "amax_out")
    if bias is not None:
        if isinstance(bias, Quantized):
            _need_operand(bias, "bias", (N,), hp_ok=False)
        else:
            _need(bias, "bias", (torch.bfloat16,), shape=(N,))
    _on_gpu(a=a, b=b, c8=c8, scale_used=scale_used, amax_out=amax_out, bias=bias)
    return (ctypes.c_int64(M), ctypes.c_int64(N), ctypes.c_int64(K), _operand(a), _operand(b),
            _operand(bias), ctypes.c_int32(fmt_out), _ring(ring_out), _vp(c8), _vp(scale_used),
            _vp(amax_out), ctypes.c_void_p(_stream(stream)))


def fp8_gemm_fp8out(a, b, c8, fmt_out, ring_out, scale_used, amax_out=None, bias=None,
                    stream=None):
    """c8 = enc_fmt_out(fl32(y * s_out)), y = a b^T / (sa sb) (+ bias) in fp32,
    s_out from ring_out (delayed scaling; folded with max |y|).  a, b:
    Quantized with contiguous codes [M, K] and [N, K]; c8: uint8 [M, N]."""
    _check(lib().fp8_gemm_fp8out(*_gemm_fp8out_args(a, b, c8, fmt_out, ring_out, scale_used,
                                                    amax_out, bias, stream)), "fp8_gemm_fp8out")


def bind_fp8_gemm_fp8out(a, b, c8, fmt_out, ring_out, scale_used, amax_out=None, bias=None,
                         stream=None):
    return _bind("fp8_gemm_fp8out", _gemm_fp8out_args(a, b, c8, fmt_out, ring_out, scale_used,
                                                      amax_out, bias, stream))


# ---------------------------------------------------------------- ragged groups, 8-bit integers
# These calls also serve single tokens, where the call itself is what takes
# time: their checks take one pass over each tensor, and sizes and pointers
# go to the C call as they are.  Every tensor must be on one GPU; the call
# runs with that GPU current, on its current stream unless one is given.

@dataclass
class QuantizedRows:
    """8-bit integer operand: int8 codes [.., rows, k] and one device float32
    scale for each row [.., rows] (a quantization multiplier: q ~ x s)."""
    codes: torch.Tensor
    scale: torch.Tensor


_F32, _U8, _I8, _I32, _BF16 = ((torch.float32,), (torch.uint8,), (torch.int8,), (torch.int32,),
                               (torch.bfloat16,))


def _gpu_of(t, what):
    t = t.codes if isinstance(t, (Quantized, QuantizedRows)) else t
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what}: expected a torch.Tensor, got {type(t).__name__}")
    return t.device


_Tensor = torch.Tensor


def _arg(t, what, dtypes, shape, dev, optional=False, numel=None):
    """Data pointer of a checked tensor argument (None when absent)."""
    if t is None and optional:
        return None
    if (isinstance(t, _Tensor) and t.dtype in dtypes and t.device == dev and t.is_cuda
            and t.is_contiguous() and (shape is None or t.shape == shape)
            and (numel is None or t.numel() >= numel)):
        return t.data_ptr()
    _need(t, what, dtypes, shape=shape, numel=numel, optional=False)
    raise ValueError(f"{what}: must be a GPU tensor on {dev} (got {t.device})")


def _shape_of(t, dims, what):
    if isinstance(t, _Tensor) and len(t.shape) == dims:
        return t.shape
    d = t.codes if isinstance(t, (Quantized, QuantizedRows)) else t
    if not isinstance(d, torch.Tensor) or d.dim() != dims:
        raise ValueError(f"{what}: expected a {dims}-D tensor")
    return d.shape


def _arg_operand(t, what, shape, dev, hp_ok=True, scales=(1,)):
    """Checked operand: a high-precision tensor, or Quantized with one of the
    given numbers of scales.  Returns (C operand, number of scales)."""
    if isinstance(t, Quantized):
        if t.fmt not in _FMT_DT:
            raise ValueError(f"{what}: unknown fp8 format {t.fmt}")
        sp = _arg(t.scale, f"{what}.scale", _F32, None, dev)
        n = t.scale.numel()
        if n not in scales:
            raise ValueError(f"{what}.scale: {n} scales, expected {' or '.join(map(str, scales))}")
        return _Operand(_arg(t.codes, f"{what}.codes", _U8, shape, dev), _FMT_DT[t.fmt], sp), n
    if not hp_ok:
        raise TypeError(f"{what}: expected a Quantized operand")
    return _Operand(_arg(t, what, _HP, shape, dev), _TORCH_DT[t.dtype], None), 1


# the current stream's handle without building a Stream object
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


# the current device without torch.cuda's check that it is initialized: the
# arguments are tensors there
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _arg_stream(stream, dev):
    if stream is None:
        return _raw_stream(dev.index)
    if stream.device != dev:
        raise ValueError(f"stream: on {stream.device}, the tensors are on {dev}")
    return stream.cuda_stream


_entry = {}  # C functions by name


def _run(name, args, dev):
    try:
        fn = _entry[name]
    except KeyError:
        fn = _entry[name] = getattr(lib(), name)
    if dev.index == _current_device():
        st = fn(*args)
    else:
        with torch.cuda.device(dev):
            st = fn(*args)
    if st != FP8_OK:
        raise Fp8Error(st, name)


def _bind_run(name, args, dev):
    return lambda: _run(name, args, dev)


_NO_OPERAND = _Operand(None, FP8_DT_BF16, None)


def _grouped_fwd_args(x, w, bias, offsets, fmt, y, ring_x, ring_w, x8_out, w8_out, sx_used,
                      sw_used, amax_x, amax_w, stream):
    T, K = _shape_of(x, 2, "x")
    E, N, Kw = _shape_of(w, 3, "w")
    dev = _gpu_of(x, "x")
    ox, _ = _arg_operand(x, "x", (T, K), dev)
    ow, ns = _arg_operand(w, "w", (E, N, K), dev, scales=(1, E))
    args = (T, E, N, K, _arg(offsets, "offsets", _I32, (E + 1,), dev), ox, ow, ns,
            _arg(bias, "bias", _BF16, (E, N), dev, True), fmt, _ring(ring_x), _ring(ring_w),
            _arg(y, "y", _BF16, (T, N), dev), _arg(x8_out, "x8_out", _U8, (T, K), dev, True),
            _arg(w8_out, "w8_out", _U8, (E, N, K), dev, True),
            _arg(sx_used, "sx_used", _F32, None, dev, True, numel=1),
            _arg(sw_used, "sw_used", _F32, None, dev, True, numel=ns),
            _arg(amax_x, "amax_x", _F32, None, dev, True, numel=1),
            _arg(amax_w, "amax_w", _F32, None, dev, True, numel=1), _arg_stream(stream, dev))
    return args, dev


def fp8_grouped_linear_fwd(x, w, bias, offsets, fmt, y, ring_x=None, ring_w=None, x8_out=None,
                           w8_out=None, sx_used=None, sw_used=None, amax_x=None, amax_w=None,
                           stream=None):
    """y[t] = x[t] w[e]^T (+ bias[e]) for the rows t of expert e, in FP8.
    x: [T, K] tensor or Quantized, rows sorted by expert; w: [E, N, K] tensor
    or Quantized with 1 or E scales; bias: bf16 [E, N] or None; offsets: int32
    [E + 1] on the GPU, expert e has rows offsets[e] .. offsets[e+1] - 1;
    y: bf16 [T, N], written in the experts' rows only."""
    _run("fp8_grouped_linear_fwd", *_grouped_fwd_args(x, w, bias, offsets, fmt, y, ring_x, ring_w,
                                                      x8_out, w8_out, sx_used, sw_used, amax_x,
                                                      amax_w, stream))


def bind_fp8_grouped_linear_fwd(x, w, bias, offsets, fmt, y, ring_x=None, ring_w=None, x8_out=None,
                                w8_out=None, sx_used=None, sw_used=None, amax_x=None, amax_w=None,
                                stream=None):
    return _bind_run("fp8_grouped_linear_fwd", *_grouped_fwd_args(
        x, w, bias, offsets, fmt, y, ring_x, ring_w, x8_out, w8_out, sx_used, sw_used, amax_x,
        amax_w, stream))


def _grouped_bwd_args(g, fmt_g, offsets, x8, w8, dx, dw, db, db_ws, ring_g, g8_out, sg_used,
                      amax_g, stream):
    T, N = _shape_of(g, 2, "g")
    dev = _gpu_of(g, "g")
    if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError("offsets: expected an int32 tensor of E + 1 elements")
    E = offsets.shape[0] - 1
    if dx is not None:
        K = _shape_of(dx, 2, "dx")[1]
    elif dw is not None:
        K = _shape_of(dw, 3, "dw")[2]
    else:
        K = 0
    og, _ = _arg_operand(g, "g", (T, N), dev)
    ox, ow, ns = _NO_OPERAND, _NO_OPERAND, 1
    if dw is not None:
        ox, _ = _arg_operand(x8, "x8", (T, K), dev, hp_ok=False)
    if dx is not None:
        ow, ns = _arg_operand(w8, "w8", (E, N, K), dev, hp_ok=False, scales=(1, E))
    wsp = None
    if db is not None and db_ws is not None:
        if not isinstance(db_ws, torch.Tensor) or not db_ws.is_contiguous():
            raise ValueError("db_ws: expected a contiguous tensor")
        if db_ws.device != dev:
            raise ValueError(f"db_ws: must be a GPU tensor on {dev} (got {db_ws.device})")
        need = fp8_grouped_db_workspace_bytes(T, E, N)
        if db_ws.numel() * db_ws.element_size() < need:
            raise ValueError(f"db_ws: {db_ws.numel() * db_ws.element_size()} bytes, "
                             f"at least {need} needed")
        wsp = db_ws.data_ptr()
        if wsp % 4:
            raise ValueError("db_ws: must be 4-byte aligned")
    args = (T, E, N, K, _arg(offsets, "offsets", _I32, (E + 1,), dev), og, fmt_g, _ring(ring_g),
            ox, ow, ns, _arg(dx, "dx", _BF16, (T, K), dev, True),
            _arg(dw, "dw", _BF16, (E, N, K), dev, True), _arg(db, "db", _BF16, (E, N), dev, True),
            wsp, _arg(g8_out, "g8_out", _U8, (T, N), dev, True),
            _arg(sg_used, "sg_used", _F32, None, dev, True, numel=1),
            _arg(amax_g, "amax_g", _F32, None, dev, True, numel=1), _arg_stream(stream, dev))
    return args, dev


def fp8_grouped_linear_bwd(g, fmt_g, offsets, x8, w8, dx=None, dw=None, db=None, db_ws=None,
                           ring_g=None, g8_out=None, sg_used=None, amax_g=None, stream=None):
    """The gradients of fp8_grouped_linear_fwd that are given a buffer: dx bf16
    [T, K] (experts' rows only), dw bf16 [E, N, K], db bf16 [E, N] (db_ws: any
    tensor of fp8_grouped_db_workspace_bytes bytes).  g: [T, N] tensor
    (quantized here) or Quantized; x8, w8: the forward's Quantized operands."""
    _run("fp8_grouped_linear_bwd", *_grouped_bwd_args(g, fmt_g, offsets, x8, w8, dx, dw, db, db_ws,
                                                      ring_g, g8_out, sg_used, amax_g, stream))


def bind_fp8_grouped_linear_bwd(g, fmt_g, offsets, x8, w8, dx=None, dw=None, db=None, db_ws=None,
                                ring_g=None, g8_out=None, sg_used=None, amax_g=None, stream=None):
    return _bind_run("fp8_grouped_linear_bwd", *_grouped_bwd_args(
        g, fmt_g, offsets, x8, w8, dx, dw, db, db_ws, ring_g, g8_out, sg_used, amax_g, stream))


def _i8_quantize_args(x, q, scale, stream):
    if not isinstance(x, torch.Tensor) or x.dim() < 1:
        raise ValueError("x: expected a tensor of at least one dimension")
    dev, cols = x.device, x.shape[-1]
    lead = x.shape[:-1]
    rows = 1
    for d in lead:
        rows *= d
    args = (_arg(x, "x", _HP, None, dev), _TORCH_DT[x.dtype], rows, cols,
            _arg(q, "q", _I8, x.shape, dev), _arg(scale, "scale", _F32, lead, dev),
            _arg_stream(stream, dev))
    return args, dev


def fp8_i8_quantize_rows(x, q, scale, stream=None):
    """q = rint(x s) with s = 127 / max |x| of each row: x [.., k], q int8 of
    x's shape, scale float32 [..]."""
    _run("fp8_i8_quantize_rows", *_i8_quantize_args(x, q, scale, stream))


def bind_fp8_i8_quantize_rows(x, q, scale, stream=None):
    return _bind_run("fp8_i8_quantize_rows", *_i8_quantize_args(x, q, scale, stream))


_OUT16 = (torch.bfloat16, torch.float16)


def _i8_rows(t, what, shape, dev):
    return _Operand(_arg(t.codes, f"{what}.codes", _I8, shape, dev), FP8_DT_I8,
                    _arg(t.scale, f"{what}.scale", _F32, shape[:-1], dev))


def _i8_args(x, w, bias, y, x8_out, sx_out, wshape, bshape, dev):
    """C arguments shared by the dense and the grouped call: x, w, bias, out
    dtype, y, x8_out, sx_out."""
    M, K = _shape_of(x, 2, "x")
    if not isinstance(w, QuantizedRows):
        raise TypeError("w: expected a QuantizedRows operand")
    yp = _arg(y, "y", _OUT16, (M, wshape[-2]), dev)
    if isinstance(x, QuantizedRows):
        ox, qp, sp = _i8_rows(x, "x", (M, K), dev), None, None
    else:
        ox = _Operand(_arg(x, "x", _HP, (M, K), dev), _TORCH_DT[x.dtype], None)
        qp = _arg(x8_out, "x8_out", _I8, (M, K), dev)
        sp = _arg(sx_out, "sx_out", _F32, None, dev, numel=M)
    return (ox, _i8_rows(w, "w", wshape, dev),
            _arg(bias, "bias", (y.dtype,), bshape, dev, True), _TORCH_DT[y.dtype], yp, qp, sp)


def _i8_linear_args(x, w, bias, y, x8_out, sx_out, stream):
    M, K = _shape_of(x, 2, "x")
    N = _shape_of(w, 2, "w")[0]
    dev = _gpu_of(x, "x")
    return (M, N, K, *_i8_args(x, w, bias, y, x8_out, sx_out, (N, K), (N,), dev),
            _arg_stream(stream, dev)), dev


def fp8_i8_linear_fwd(x, w, bias, y, x8_out=None, sx_out=None, stream=None):
    """y = x w^T (+ bias) in 8-bit integers, a scale for each token and output
    channel.  x: [M, K] tensor (quantized here into x8_out int8 [M, K] and
    sx_out float32 [M]) or QuantizedRows; w: QuantizedRows [N, K]; y bf16 or
    fp16 [M, N]; bias of y's dtype [N] or None."""
    _run("fp8_i8_linear_fwd", *_i8_linear_args(x, w, bias, y, x8_out, sx_out, stream))


def bind_fp8_i8_linear_fwd(x, w, bias, y, x8_out=None, sx_out=None, stream=None):
    return _bind_run("fp8_i8_linear_fwd", *_i8_linear_args(x, w, bias, y, x8_out, sx_out, stream))


def _i8_grouped_args(x, w, bias, offsets, y, x8_out, sx_out, stream):
    T, K = _shape_of(x, 2, "x")
    E, N, _ = _shape_of(w, 3, "w")
    dev = _gpu_of(x, "x")
    return (T, E, N, K, _arg(offsets, "offsets", _I32, (E + 1,), dev),
            *_i8_args(x, w, bias, y, x8_out, sx_out, (E, N, K), (E, N), dev),
            _arg_stream(stream, dev)), dev


def fp8_i8_grouped_linear_fwd(x, w, bias, offsets, y, x8_out=None, sx_out=None, stream=None):
    """fp8_i8_linear_fwd over experts: w QuantizedRows [E, N, K] (scales
    [E, N]), bias [E, N], offsets as in fp8_grouped_linear_fwd.  Rows behind
    the last expert's are left as they were in y, x8_out and sx_out."""
    _run("fp8_i8_grouped_linear_fwd", *_i8_grouped_args(x, w, bias, offsets, y, x8_out, sx_out,
                                                        stream))


def bind_fp8_i8_grouped_linear_fwd(x, w, bias, offsets, y, x8_out=None, sx_out=None, stream=None):
    return _bind_run("fp8_i8_grouped_linear_fwd", *_i8_grouped_args(x, w, bias, offsets, y, x8_out,
                                                                    sx_out, stream))


# ---------------------------------------------------------------- 4-bit floating point

@dataclass
class QuantizedMx4:
    """Operand in microscaled 4-bit floating point: uint8 codes
    [.., rows, 16 ceil(k / 32)] (two to a byte), uint8 scales
    [.., ceil(k / 128), rows, 4] (biased exponents, four blocks of 32 values to
    a word), and k, the values in a row."""
    codes: torch.Tensor
    scale: torch.Tensor
    cols: int

    @staticmethod
    def empty(*shape, device="cuda"):
        """Buffers for a matrix, or a stack of matrices, of the given shape."""
        *lead, rows, k = shape
        return QuantizedMx4(
            torch.empty(*lead, rows, 16 * (-(-k // 32)), dtype=torch.uint8, device=device),
            torch.empty(*lead, -(-k // 128), rows, 4, dtype=torch.uint8, device=device), k)


def _mx4_shapes(lead, rows, k):
    return (*lead, rows, 16 * (-(-k // 32))), (*lead, -(-k // 128), rows, 4)


def _mx4_pointers(codes, scales, what, lead, rows, k, dev):
    sc, ss = _mx4_shapes(lead, rows, k)
    return _arg(codes, f"{what}.codes", _U8, sc, dev), _arg(scales, f"{what}.scale", _U8, ss, dev)


def _mx4_quantize_args(x, codes, scales, stream):
    if not isinstance(x, torch.Tensor) or x.dim() < 2:
        raise ValueError("x: expected a matrix or a stack of matrices")
    dev, (*lead, rows, k) = x.device, x.shape
    mats = 1
    for d in lead:
        mats *= d
    return (_arg(x, "x", _HP, None, dev), _TORCH_DT[x.dtype], mats, rows, k,
            *_mx4_pointers(codes, scales, "out", lead, rows, k, dev), _arg_stream(stream, dev)), dev


def fp8_mx4_quantize(x, codes, scales, stream=None):
    """x [.., rows, k] to 4-bit codes and block exponents (the buffers of
    QuantizedMx4.empty(*x.shape))."""
    _run("fp8_mx4_quantize", *_mx4_quantize_args(x, codes, scales, stream))


def bind_fp8_mx4_quantize(x, codes, scales, stream=None):
    return _bind_run("fp8_mx4_quantize", *_mx4_quantize_args(x, codes, scales, stream))


def _mx4_dequantize_args(q, out, stream):
    if not isinstance(q, QuantizedMx4):
        raise TypeError("q: expected a QuantizedMx4 operand")
    if not isinstance(out, torch.Tensor) or out.dim() < 2:
        raise ValueError("out: expected a matrix or a stack of matrices")
    dev, (*lead, rows, k) = out.device, out.shape
    if k != q.cols:
        raise ValueError(f"out: rows of {k} values, q has {q.cols}")
    mats = 1
    for d in lead:
        mats *= d
    return (*_mx4_pointers(q.codes, q.scale, "q", lead, rows, k, dev), mats, rows, k,
            _arg(out, "out", _HP, None, dev), _TORCH_DT[out.dtype], _arg_stream(stream, dev)), dev


def fp8_mx4_dequantize(q, out, stream=None):
    """The values of q (QuantizedMx4), rounded once to out's type."""
    _run("fp8_mx4_dequantize", *_mx4_dequantize_args(q, out, stream))


def bind_fp8_mx4_dequantize(q, out, stream=None):
    return _bind_run("fp8_mx4_dequantize", *_mx4_dequantize_args(q, out, stream))


def _mx4_args(x, w, bias, y, x4_out, sx_out, lead, M, N, dev):
    """C arguments shared by the dense and the grouped call: x, its type and
    scales, w and its scales, bias, out dtype, y, x4_out, sx_out."""
    k = w.cols
    cb, sb = 16 * (-(-k // 32)), -(-k // 128)  # of a row, as _mx4_shapes has them
    if isinstance(x, QuantizedMx4):
        if x.cols != k:
            raise ValueError(f"x: rows of {x.cols} values, w has {k}")
        xp, xs = _mx4_pointers(x.codes, x.scale, "x", (), M, k, dev)
        dt, qp, sp = FP8_DT_MX4, None, None
    else:
        xp, xs, dt = _arg(x, "x", _HP, (M, k), dev), None, _TORCH_DT[x.dtype]
        qp = _arg(x4_out, "x4_out", _U8, (M, cb), dev)
        sp = _arg(sx_out, "sx_out", _U8, (sb, M, 4), dev)
    yp = _arg(y, "y", _OUT16, (M, N), dev)
    return (xp, dt, xs, _arg(w.codes, "w.codes", _U8, (*lead, N, cb), dev),
            _arg(w.scale, "w.scale", _U8, (*lead, sb, N, 4), dev),
            None if bias is None else _arg(bias, "bias", (y.dtype,), (*lead, N), dev),
            _TORCH_DT[y.dtype], yp, qp, sp)


def _mx4_linear_args(x, w, bias, y, x4_out, sx_out, stream):
    if not isinstance(w, QuantizedMx4):
        raise TypeError("w: expected a QuantizedMx4 operand")
    N = _shape_of(w.codes, 2, "w.codes")[0]
    xc = x.codes if isinstance(x, QuantizedMx4) else x
    M = _shape_of(xc, 2, "x")[0]
    dev = xc.device
    return (M, N, w.cols, *_mx4_args(x, w, bias, y, x4_out, sx_out, (), M, N, dev),
            _arg_stream(stream, dev)), dev


def fp8_mx4_linear_fwd(x, w, bias, y, x4_out=None, sx_out=None, stream=None):
    """y = x w^T (+ bias) in 4-bit floating point.  x: [M, k] tensor (quantized
    here into x4_out and sx_out, the buffers of QuantizedMx4.empty(M, k)) or
    QuantizedMx4; w: QuantizedMx4 of [N, k]; y bf16 or fp16 [M, N]; bias of y's
    dtype [N] or None."""
    _run("fp8_mx4_linear_fwd", *_mx4_linear_args(x, w, bias, y, x4_out, sx_out, stream))


def bind_fp8_mx4_linear_fwd(x, w, bias, y, x4_out=None, sx_out=None, stream=None):
    return _bind_run("fp8_mx4_linear_fwd", *_mx4_linear_args(x, w, bias, y, x4_out, sx_out, stream))


def _mx4_grouped_args(x, w, bias, offsets, y, x4_out, sx_out, stream):
    if not isinstance(w, QuantizedMx4):
        raise TypeError("w: expected a QuantizedMx4 operand")
    E, N, _ = _shape_of(w.codes, 3, "w.codes")
    xc = x.codes if isinstance(x, QuantizedMx4) else x
    T = _shape_of(xc, 2, "x")[0]
    dev = xc.device
    return (T, E, N, w.cols, _arg(offsets, "offsets", _I32, (E + 1,), dev),
            *_mx4_args(x, w, bias, y, x4_out, sx_out, (E,), T, N, dev),
            _arg_stream(stream, dev)), dev


def fp8_mx4_grouped_linear_fwd(x, w, bias, offsets, y, x4_out=None, sx_out=None, stream=None):
    """fp8_mx4_linear_fwd over experts: w QuantizedMx4 of [E, N, k], bias
    [E, N], offsets as in fp8_grouped_linear_fwd.  Rows behind the last
    expert's are left as they were in y, x4_out and sx_out."""
    _run("fp8_mx4_grouped_linear_fwd", *_mx4_grouped_args(x, w, bias, offsets, y, x4_out, sx_out,
                                                          stream))


def bind_fp8_mx4_grouped_linear_fwd(x, w, bias, offsets, y, x4_out=None, sx_out=None, stream=None):
    return _bind_run("fp8_mx4_grouped_linear_fwd", *_mx4_grouped_args(x, w, bias, offsets, y,
                                                                      x4_out, sx_out, stream))


# ---------------------------------------------------------------- routing to experts

def _arg_places(T, k, E, offsets, pos, ws, dev):
    """Pointers of a call that places rows: offsets, pos, workspace."""
    op = _arg(offsets, "offsets", _I32, (E + 1,), dev)
    pp = _arg(pos, "pos", _I32, (T, k), dev)
    if ws is None:  # the library refuses it where it needs one
        return op, pp, None
    need = fp8_route_workspace_bytes(T, E, k)
    if need == 0:
        return op, pp, None
    if not isinstance(ws, torch.Tensor) or not ws.is_contiguous():
        raise ValueError(f"ws: expected a contiguous tensor of {need} bytes")
    if ws.device != dev:
        raise ValueError(f"ws: must be a GPU tensor on {dev} (got {ws.device})")
    if ws.numel() * ws.element_size() < need:
        raise ValueError(f"ws: {ws.numel() * ws.element_size()} bytes, at least {need} needed")
    if ws.data_ptr() % 4:
        raise ValueError("ws: must be 4-byte aligned")
    return op, pp, ws.data_ptr()


def _route_fwd_args(logits, idx, weights, bias, score, groups, groups_kept, group_top, renorm,
                    scale, offsets, pos, ws, stream):
    T, E = _shape_of(logits, 2, "logits")
    k = _shape_of(idx, 2, "idx")[1]
    dev = logits.device
    zp = _arg(logits, "logits", _HP, None, dev)
    places = (None, None, None)
    if offsets is not None or pos is not None:
        places = _arg_places(T, k, E, offsets, pos, ws, dev)
    return (T, E, k, zp, _TORCH_DT[logits.dtype], _arg(bias, "bias", _F32, (E,), dev, True), score,
            groups, groups_kept, group_top, int(bool(renorm)), scale,
            _arg(idx, "idx", _I32, (T, k), dev), _arg(weights, "weights", _F32, (T, k), dev),
            *places, _arg_stream(stream, dev)), dev


def fp8_route_fwd(logits, idx, weights, bias=None, score=FP8_ROUTE_SOFTMAX, groups=1,
                  groups_kept=1, group_top=1, renorm=True, scale=1.0, offsets=None, pos=None,
                  ws=None, stream=None):
    """The k experts of each token and their weights: logits [T, E], idx int32
    [T, k], weights float32 [T, k], bias float32 [E] or None (added to the
    scores for the choice only).  With offsets int32 [E + 1] and pos int32
    [T, k] also the places of the rows sorted by expert (ws: any tensor of
    fp8_route_workspace_bytes bytes, None where that is 0)."""
    _run("fp8_route_fwd", *_route_fwd_args(logits, idx, weights, bias, score, groups, groups_kept,
                                           group_top, renorm, scale, offsets, pos, ws, stream))


def bind_fp8_route_fwd(logits, idx, weights, bias=None, score=FP8_ROUTE_SOFTMAX, groups=1,
                       groups_kept=1, group_top=1, renorm=True, scale=1.0, offsets=None, pos=None,
                       ws=None, stream=None):
    return _bind_run("fp8_route_fwd", *_route_fwd_args(
        logits, idx, weights, bias, score, groups, groups_kept, group_top, renorm, scale, offsets,
        pos, ws, stream))


def _route_bwd_args(logits, idx, dweights, dlogits, score, renorm, scale, stream):
    T, E = _shape_of(logits, 2, "logits")
    k = _shape_of(idx, 2, "idx")[1]
    dev = logits.device
    return (T, E, k, _arg(logits, "logits", _HP, None, dev), _TORCH_DT[logits.dtype], score,
            int(bool(renorm)), scale, _arg(idx, "idx", _I32, (T, k), dev),
            _arg(dweights, "dweights", _F32, (T, k), dev),
            _arg(dlogits, "dlogits", (logits.dtype,), (T, E), dev), _arg_stream(stream, dev)), dev


def fp8_route_bwd(logits, idx, dweights, dlogits, score=FP8_ROUTE_SOFTMAX, renorm=True, scale=1.0,
                  stream=None):
    """dlogits [T, E] (of logits' type) from dweights float32 [T, k] and the
    forward's logits, idx and settings."""
    _run("fp8_route_bwd", *_route_bwd_args(logits, idx, dweights, dlogits, score, renorm, scale,
                                           stream))


def bind_fp8_route_bwd(logits, idx, dweights, dlogits, score=FP8_ROUTE_SOFTMAX, renorm=True,
                       scale=1.0, stream=None):
    return _bind_run("fp8_route_bwd", *_route_bwd_args(logits, idx, dweights, dlogits, score,
                                                       renorm, scale, stream))


def _route_plan_args(idx, offsets, pos, ws, stream):
    T, k = _shape_of(idx, 2, "idx")
    E = _shape_of(offsets, 1, "offsets")[0] - 1
    dev = idx.device
    return (T, E, k, _arg(idx, "idx", _I32, None, dev),
            *_arg_places(T, k, E, offsets, pos, ws, dev), _arg_stream(stream, dev)), dev


def fp8_route_plan(idx, offsets, pos, ws=None, stream=None):
    """Places of the rows sorted by expert, of idx int32 [T, k] from anywhere:
    offsets int32 [E + 1], pos int32 [T, k] (-1: no expert)."""
    _run("fp8_route_plan", *_route_plan_args(idx, offsets, pos, ws, stream))


def bind_fp8_route_plan(idx, offsets, pos, ws=None, stream=None):
    return _bind_run("fp8_route_plan", *_route_plan_args(idx, offsets, pos, ws, stream))


def _route_gather_args(x, pos, out, stream):
    T, D = _shape_of(x, 2, "x")
    k = _shape_of(pos, 2, "pos")[1]
    R = _shape_of(out, 2, "out")[0]
    dev = x.device
    return (T, k, D * x.element_size(), R, _arg(x, "x", (x.dtype,), None, dev),
            _arg(pos, "pos", _I32, (T, k), dev), _arg(out, "out", (x.dtype,), (R, D), dev),
            _arg_stream(stream, dev)), dev


def fp8_route_gather(x, pos, out, stream=None):
    """out[pos[t, i]] = x[t]: x [T, D] and out [R, D] of one type, whichever
    (values, codes, scales).  Rows of out that no slot names stay as they
    were."""
    _run("fp8_route_gather", *_route_gather_args(x, pos, out, stream))


def bind_fp8_route_gather(x, pos, out, stream=None):
    return _bind_run("fp8_route_gather", *_route_gather_args(x, pos, out, stream))


def _route_combine_args(y, pos, weights, out, stream):
    R, D = _shape_of(y, 2, "y")
    T, k = _shape_of(pos, 2, "pos")
    dev = y.device
    yp = _arg(y, "y", _HP, None, dev)
    return (T, k, D, R, yp, _TORCH_DT[y.dtype], _arg(pos, "pos", _I32, None, dev),
            _arg(weights, "weights", _F32, (T, k), dev, True),
            _arg(out, "out", (y.dtype,), (T, D), dev), _arg_stream(stream, dev)), dev


def fp8_route_combine(y, pos, weights, out, stream=None):
    """out[t] = sum_i weights[t, i] y[pos[t, i]]: y [R, D], out [T, D] of y's
    type, weights float32 [T, k] or None (ones: the gradient of
    fp8_route_gather)."""
    _run("fp8_route_combine", *_route_combine_args(y, pos, weights, out, stream))


def bind_fp8_route_combine(y, pos, weights, out, stream=None):
    return _bind_run("fp8_route_combine", *_route_combine_args(y, pos, weights, out, stream))


def _route_combine_bwd_args(dout, y, pos, weights, dy, dweights, stream):
    T, D = _shape_of(dout, 2, "dout")
    k = _shape_of(pos, 2, "pos")[1]
    dev = dout.device
    gp = _arg(dout, "dout", _HP, None, dev)
    R = _shape_of(dy if y is None else y, 2, "y")[0]
    dt = (dout.dtype,)
    return (T, k, D, R, gp, _arg(y, "y", dt, (R, D), dev, dweights is None), _TORCH_DT[dout.dtype],
            _arg(pos, "pos", _I32, (T, k), dev), _arg(weights, "weights", _F32, (T, k), dev),
            _arg(dy, "dy", dt, (R, D), dev, True),
            _arg(dweights, "dweights", _F32, (T, k), dev, True), _arg_stream(stream, dev)), dev


def fp8_route_combine_bwd(dout, y, pos, weights, dy=None, dweights=None, stream=None):
    """The gradients of fp8_route_combine that are given a buffer:
    dy[pos[t, i]] = weights[t, i] dout[t] (other rows stay as they were) and
    dweights[t, i] = dout[t] . y[pos[t, i]] (y is needed for these only)."""
    _run("fp8_route_combine_bwd", *_route_combine_bwd_args(dout, y, pos, weights, dy, dweights,
                                                           stream))


def bind_fp8_route_combine_bwd(dout, y, pos, weights, dy=None, dweights=None, stream=None):
    return _bind_run("fp8_route_combine_bwd", *_route_combine_bwd_args(dout, y, pos, weights, dy,
                                                                       dweights, stream))
