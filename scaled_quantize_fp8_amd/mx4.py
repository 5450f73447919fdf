"""Serving modules over the 4-bit floating point linear layers: weights
quantized once in blocks of 32 along K, activations in every call.  Every step
of the computation runs in the library; these modules hold the codes and
allocate outputs.
"""

from __future__ import annotations

import torch

from . import (QuantizedMx4, fp8_mx4_dequantize, fp8_mx4_grouped_linear_fwd, fp8_mx4_linear_fwd,
               fp8_mx4_quantize)


def _no_grad(x):
    if torch.is_grad_enabled() and x.requires_grad:
        raise RuntimeError("4-bit layers serve a trained model: they have no gradient")


class _Mx4Weights(torch.nn.Module):
    """Codes and block exponents of weight [.., N, K] (bf16, fp16 or fp32, on
    the GPU) and the bias [.., N] in the output's type."""

    def __init__(self, weight, bias=None, out_dtype=torch.bfloat16):
        super().__init__()
        w = weight.detach().contiguous()
        q = QuantizedMx4.empty(*w.shape, device=w.device)
        fp8_mx4_quantize(w, q.codes, q.scale)
        self.in_features, self.out_features, self.out_dtype = w.shape[-1], w.shape[-2], out_dtype
        self.register_buffer("codes", q.codes)
        self.register_buffer("scale", q.scale)
        self.register_buffer("bias", None if bias is None else
                             bias.detach().to(out_dtype).contiguous())

    def _weight(self):
        return QuantizedMx4(self.codes, self.scale, self.in_features)

    def _buffers_for(self, x2):
        q = QuantizedMx4.empty(*x2.shape, device=x2.device)
        return q.codes, q.scale

    def dequantize(self, dtype=torch.bfloat16):
        """The weight [.., N, K] that the codes stand for."""
        w = torch.empty(*self.codes.shape[:-1], self.in_features, dtype=dtype,
                        device=self.codes.device)
        fp8_mx4_dequantize(self._weight(), w)
        return w


class Mx4Linear(_Mx4Weights):
    """y = x W^T + b in 4-bit floating point; x [.., K] bf16, fp16 or fp32."""

    @classmethod
    def from_linear(cls, lin, out_dtype=torch.bfloat16):
        """Of a layer with ``weight`` [N, K] and ``bias`` [N] or None
        (torch.nn.Linear, Fp8Linear)."""
        return cls(lin.weight, lin.bias, out_dtype)

    def forward(self, x):
        _no_grad(x)
        x2 = x.reshape(-1, x.shape[-1]).contiguous()
        y = torch.empty(x2.shape[0], self.out_features, dtype=self.out_dtype, device=x.device)
        fp8_mx4_linear_fwd(x2, self._weight(), self.bias, y, *self._buffers_for(x2))
        return y.view(*x.shape[:-1], y.shape[-1])


class Mx4GroupedLinear(_Mx4Weights):
    """y[t] = x[t] W[e]^T + b[e] for the rows t of expert e in 4-bit floating
    point; x [T, K] with rows sorted by expert, offsets int32 [E + 1] on the
    GPU.  Rows of no expert give zeros."""

    @classmethod
    def from_grouped(cls, lin, out_dtype=torch.bfloat16):
        """Of an Fp8GroupedLinear."""
        return cls(lin.weight, lin.bias, out_dtype)

    def forward(self, x, offsets):
        _no_grad(x)
        x = x.contiguous()
        y = torch.zeros(x.shape[0], self.out_features, dtype=self.out_dtype, device=x.device)
        fp8_mx4_grouped_linear_fwd(x, self._weight(), self.bias, offsets, y,
                                   *self._buffers_for(x))
        return y
