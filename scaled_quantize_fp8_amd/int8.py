"""Serving modules over the 8-bit integer linear layers: weights quantized
once by output channel, activations by token in every call.  Every step of
the computation runs in the library; these modules hold the codes and
allocate outputs.
"""

from __future__ import annotations

import torch

from . import (QuantizedRows, fp8_i8_grouped_linear_fwd, fp8_i8_linear_fwd, fp8_i8_quantize_rows)


def _no_grad(x):
    if torch.is_grad_enabled() and x.requires_grad:
        raise RuntimeError("8-bit integer layers serve a trained model: they have no gradient")


class _Int8Weights(torch.nn.Module):
    """Codes and scales of weight [.., N, K] (bf16, fp16 or fp32, on the GPU)
    and the bias [.., N] in the output's type."""

    def __init__(self, weight, bias=None, out_dtype=torch.bfloat16):
        super().__init__()
        w = weight.detach().contiguous()
        codes = torch.empty(w.shape, dtype=torch.int8, device=w.device)
        scale = torch.empty(w.shape[:-1], dtype=torch.float32, device=w.device)
        fp8_i8_quantize_rows(w, codes, scale)
        self.out_dtype = out_dtype
        self.register_buffer("codes", codes)
        self.register_buffer("scale", scale)
        self.register_buffer("bias", None if bias is None else
                             bias.detach().to(out_dtype).contiguous())

    def _buffers_for(self, x2):
        M, K = x2.shape
        return (torch.empty(M, K, dtype=torch.int8, device=x2.device),
                torch.empty(M, dtype=torch.float32, device=x2.device))


class Int8Linear(_Int8Weights):
    """y = x W^T + b in 8-bit integers; x [.., K] bf16, fp16 or fp32."""

    @classmethod
    def from_linear(cls, lin, out_dtype=torch.bfloat16):
        """Of a layer with ``weight`` [N, K] and ``bias`` [N] or None
        (torch.nn.Linear, Fp8Linear)."""
        return cls(lin.weight, lin.bias, out_dtype)

    def forward(self, x):
        _no_grad(x)
        x2 = x.reshape(-1, x.shape[-1]).contiguous()
        y = torch.empty(x2.shape[0], self.codes.shape[0], dtype=self.out_dtype, device=x.device)
        fp8_i8_linear_fwd(x2, QuantizedRows(self.codes, self.scale), self.bias, y,
                          *self._buffers_for(x2))
        return y.view(*x.shape[:-1], y.shape[-1])


class Int8GroupedLinear(_Int8Weights):
    """y[t] = x[t] W[e]^T + b[e] for the rows t of expert e in 8-bit integers;
    x [T, K] with rows sorted by expert, offsets int32 [E + 1] on the GPU.
    Rows of no expert give zeros."""

    @classmethod
    def from_grouped(cls, lin, out_dtype=torch.bfloat16):
        """Of an Fp8GroupedLinear."""
        return cls(lin.weight, lin.bias, out_dtype)

    def forward(self, x, offsets):
        _no_grad(x)
        x = x.contiguous()
        y = torch.zeros(x.shape[0], self.codes.shape[1], dtype=self.out_dtype, device=x.device)
        fp8_i8_grouped_linear_fwd(x, QuantizedRows(self.codes, self.scale), self.bias, offsets, y,
                                  *self._buffers_for(x))
        return y
