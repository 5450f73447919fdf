"""torch.autograd wrappers of the routing to experts and of the exchange of
rows with them, and a mixture of experts made of those and of the grouped
linear layers.

route gives every token its experts, their weights and the places of its rows
when rows are sorted by expert; dispatch copies tokens there; combine brings
the experts' rows back as weighted sums.  The choice of experts has no
gradient: the weights' goes to the logits, and to no bias.  Every step of the
computation runs in the library; this module allocates outputs and marshals
arguments.
"""

from __future__ import annotations

import torch

from . import (FP8_ROUTE_SIGMOID, FP8_ROUTE_SOFTMAX, fp8_route_bwd, fp8_route_combine,
               fp8_route_combine_bwd, fp8_route_fwd, fp8_route_gather, fp8_route_workspace_bytes)
from .autograd import Fp8GroupedLinear

_SCORES = {"softmax": FP8_ROUTE_SOFTMAX, "sigmoid": FP8_ROUTE_SIGMOID}


def _one_stream(out):
    """out, a result of a call whose inputs may be leaves.  Autograd brings a
    leaf's gradient to the stream on which the leaf's oldest living graph was
    built; a backward captured on another stream would draw that one into the
    capture, which ends the process when the capture does.  So the stream is
    noted at the leaf's node, which lives as long as such a graph, and a
    captured call that meets another one is refused."""
    if out.grad_fn is not None:
        here = torch.cuda.current_stream(out.device).cuda_stream
        for node, _ in out.grad_fn.next_functions:
            if node is None or node.name() != "torch::autograd::AccumulateGrad":
                continue
            if (node.metadata.setdefault("fp8linear.stream", here) != here
                    and torch.cuda.is_current_stream_capturing()):
                raise RuntimeError("captured beside a living eager graph of the same leaves on "
                                   "another stream: drop that graph's outputs first")
    return out


class _RouteFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, bias, k, score, groups, groups_kept, group_top, renorm, scale):
        z = logits.contiguous()
        T, E = z.shape
        dev = z.device
        idx = torch.empty(T, k, dtype=torch.int32, device=dev)
        weights = torch.empty(T, k, dtype=torch.float32, device=dev)
        offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
        pos = torch.empty(T, k, dtype=torch.int32, device=dev)
        need = fp8_route_workspace_bytes(T, E, k)
        ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
        fp8_route_fwd(z, idx, weights, bias, score, groups, groups_kept, group_top, renorm, scale,
                      offsets, pos, ws)
        ctx.save_for_backward(z, idx)
        ctx.how = (score, renorm, scale)
        ctx.mark_non_differentiable(idx, pos, offsets)
        return weights, idx, pos, offsets

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dweights, _idx, _pos, _offsets):
        z, idx = ctx.saved_tensors
        dz = torch.empty_like(z)
        fp8_route_bwd(z, idx, dweights.float().contiguous(), dz, *ctx.how)
        return (dz,) + (None,) * 8


def route(logits, k, bias=None, score="softmax", groups=1, groups_kept=1, group_top=1,
          renorm=True, scale=1.0):
    """The k experts of each row of logits [T, E] (bf16, fp16 or fp32):
    weights float32 [T, k] (with a gradient), experts int32 [T, k] (-1: none),
    and for rows sorted by expert their places pos int32 [T, k] and offsets
    int32 [E + 1].  score: "softmax" or "sigmoid"; bias float32 [E] is added to
    the scores for the choice only; of ``groups`` equal runs of experts only
    the groups_kept with the largest sums of their group_top best are chosen
    from; renorm divides a row's weights by their sum; scale multiplies them."""
    if score not in _SCORES:
        raise ValueError(f"score: expected one of {sorted(_SCORES)} (got {score!r})")
    out = _RouteFn.apply(logits, bias, k, _SCORES[score], groups, groups_kept, group_top, renorm,
                         scale)
    _one_stream(out[0])
    return out


class _DispatchFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, pos):
        x = x.contiguous()
        # zeros: places that no slot names are not written
        xs = torch.zeros(pos.numel(), x.shape[1], dtype=x.dtype, device=x.device)
        fp8_route_gather(x, pos, xs)
        ctx.save_for_backward(pos)
        return xs

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dxs):
        pos, = ctx.saved_tensors
        dx = torch.empty(pos.shape[0], dxs.shape[1], dtype=dxs.dtype, device=dxs.device)
        fp8_route_combine(dxs.contiguous(), pos, None, dx)
        return dx, None


def dispatch(x, pos):
    """Rows in expert order: xs[pos[t, i]] = x[t], [T k, D] from [T, D].  Rows
    of no expert, behind the last expert's, are zeros."""
    return _one_stream(_DispatchFn.apply(x, pos))


class _CombineFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ys, pos, weights):
        ys, weights = ys.contiguous(), weights.contiguous()
        out = torch.empty(pos.shape[0], ys.shape[1], dtype=ys.dtype, device=ys.device)
        fp8_route_combine(ys, pos, weights, out)
        ctx.save_for_backward(ys, pos, weights)
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        ys, pos, weights = ctx.saved_tensors
        need_y, _, need_w = ctx.needs_input_grad
        # zeros: places that no slot names are not written
        dys = torch.zeros_like(ys) if need_y else None
        dw = torch.empty_like(weights) if need_w else None
        fp8_route_combine_bwd(dout.contiguous(), ys, pos, weights, dys, dw)
        return dys, None, dw


def combine(ys, pos, weights):
    """out[t] = sum_i weights[t, i] ys[pos[t, i]]: ys [R, D], weights float32
    [T, k]."""
    return _one_stream(_CombineFn.apply(ys, pos, weights))


class Router(torch.nn.Module):
    """route of the logits x W^T (x bf16 [T, in], W bf16 [experts, in]; the
    logits are rounded to bf16), with the settings of ``route``.  With
    ``bias`` a float32 buffer [experts] of zeros is added to the scores for
    the choice; it gets no gradient, a training loop that balances the
    experts' loads sets it."""

    def __init__(self, in_features: int, experts: int, k: int, bias: bool = False, device=None,
                 **how):
        super().__init__()
        self.in_features, self.experts, self.k, self.how = in_features, experts, k, how
        self.weight = torch.nn.Parameter(torch.empty(experts, in_features, dtype=torch.bfloat16,
                                                     device=device))
        torch.nn.init.normal_(self.weight, std=0.02)
        self.register_buffer("bias", torch.zeros(experts, dtype=torch.float32, device=device)
                             if bias else None)

    def forward(self, x):
        _one_stream(weight := self.weight.view_as(self.weight))
        return route(torch.nn.functional.linear(x, weight), self.k, self.bias, **self.how)


class Mixture(torch.nn.Module):
    """A mixture of feed-forward experts: y[t] = sum_i w[t, i] f_e(x[t]) over
    the k experts e of token t, f_e(x) = down_e(gelu(up_e(x))).  x bf16 [.., d].
    The layers train in FP8 (Fp8GroupedLinear); ``served`` replaces them."""

    def __init__(self, d: int, ffn: int, experts: int, k: int, device=None, **how):
        super().__init__()
        self.router = Router(d, experts, k, device=device, **how)
        self.up = Fp8GroupedLinear(experts, d, ffn, device=device)
        self.down = Fp8GroupedLinear(experts, ffn, d, device=device)

    def forward(self, x):
        x2 = x.reshape(-1, x.shape[-1])
        weights, _, pos, offsets = self.router(x2)
        h = torch.nn.functional.gelu(_one_stream(self.up(dispatch(x2, pos), offsets)))
        return combine(_one_stream(self.down(h, offsets)), pos, weights).view(x.shape)

    def served(self, grouped):
        """The same mixture over layers of another kind: grouped is
        Mx4GroupedLinear or Int8GroupedLinear.  The router is shared."""
        mix = Mixture.__new__(Mixture)
        torch.nn.Module.__init__(mix)
        mix.router = self.router
        mix.up, mix.down = grouped.from_grouped(self.up), grouped.from_grouped(self.down)
        return mix
