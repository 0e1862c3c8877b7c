"""The pieces of a MoE block around its experts' products, as PyTorch functions.

``rms_norm``, ``moe_route`` and ``moe_combine`` are the autograd forms of ``rmsnorm``, ``route`` and
``combine``: every arithmetic step runs in libnvfp4's kernels, this module only sequences the calls and keeps
what the backward pass reads.  ``expert_gemv`` and, with the activation inside, ``expert_mlp`` are the experts'
forward pass for the few tokens of a decoding step, on the NVFP4 weights that ``grouped_gemm`` uses for many.

    y, h = rms_norm(x, norm_weight, residual)          # h: the residual stream
    r = moe_route(y.float() @ router.t(), top_k=4)     # experts, weights, the rows' order
    out = expert_mlp(y, r, up, down, gate, base=h)     # decoding; or, with gradients of rows and weights,
    out = moe_combine(rows, r, base=h)

Gradients cannot be captured into a CUDA graph through these functions: a leaf whose gradient an eager graph
still accumulates on another stream would tie that stream into the capture.  They refuse it; capture the
``*_backward`` calls of the package instead, which take and return plain tensors.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import (NVFP4_OUT_BF16, NVFP4_OUT_F32, Routing, combine, combine_backward, expert_mlp as _expert_mlp,
               grouped_gemv, rmsnorm, rmsnorm_backward, route, route_backward)


def _refuse_captured_gradients(name: str, *tensors) -> None:
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors):
        _refuse_capture(name)


def _refuse_capture(name: str) -> None:
    if torch.cuda.is_available() and torch.cuda.is_current_stream_capturing():
        raise RuntimeError(f"{name}: gradients cannot be captured into a CUDA graph through autograd; capture the "
                           f"package's forward and backward calls")


def _gradient(t):
    """A gradient as the kernels read it: contiguous rows from a 16-byte boundary (a piece of a larger tensor may
    begin anywhere)."""
    if t is None:
        return None
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


class _RMSNorm(torch.autograd.Function):
    # x and residual come in their own shapes: views of their gradient, one for each, would be taken for tensors of
    # their own, and two leaves would accumulate into the same memory
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        cols = x.shape[-1]
        f = rmsnorm(x.reshape(-1, cols), weight, None if residual is None else residual.reshape(-1, cols), eps,
                    rstd=True)
        ctx.save_for_backward(x if residual is None else f["h"], weight, f["rstd"])
        ctx.shape = x.shape
        ctx.has_residual = residual is not None
        ctx.set_materialize_grads(False)
        return (f["y"], f["h"]) if residual is not None else f["y"]

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, dh=None):
        _refuse_capture("rms_norm")
        h, weight, rstd = ctx.saved_tensors
        if dy is None:  # only the sum was used
            dx, dw = dh.clone(memory_format=torch.contiguous_format), None
        else:
            dx, dw = rmsnorm_backward(_gradient(dy), h.reshape(-1, ctx.shape[-1]), weight, rstd, _gradient(dh),
                                      dweight=ctx.needs_input_grad[1])
        dx = dx.view(ctx.shape)
        return dx, dw, dx if ctx.has_residual else None, None


def rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, eps: float = 1e-6):
    """Root-mean-square norm of x [..., cols] times weight [cols].  With a residual of x's shape: (y, h), the norm
    of h = x + residual and h itself; without: y.  x and residual bf16, weight bf16 or f32."""
    _refuse_captured_gradients("rms_norm", x, weight, residual)
    if residual is None:
        return _RMSNorm.apply(x, weight, None, eps).reshape(x.shape)
    if residual.shape != x.shape:
        raise ValueError(f"rms_norm: residual {tuple(residual.shape)} and x {tuple(x.shape)} differ")
    y, h = _RMSNorm.apply(x, weight, residual, eps)
    return y.reshape(x.shape), h.reshape(x.shape)


class RMSNorm(torch.nn.Module):
    """``rms_norm`` with a learned weight (bf16 by default), starting at one."""

    def __init__(self, cols: int, eps: float = 1e-6, device=None, dtype=torch.bfloat16):
        super().__init__()
        self.eps = eps
        self.weight = torch.nn.Parameter(torch.ones(cols, dtype=dtype, device=device))

    def forward(self, x: torch.Tensor, residual: torch.Tensor | None = None):
        return rms_norm(x, self.weight, residual, self.eps)


class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, top_k, options, kept):
        r = route(logits, top_k, **options)
        kept.append(r.params)
        ctx.save_for_backward(logits, r.expert)
        ctx.params = r.params
        ctx.mark_non_differentiable(r.expert, r.group_offsets, r.row_index, r.slot_row)
        return r.weight, r.expert, r.group_offsets, r.row_index, r.slot_row

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dweight, *_):
        _refuse_capture("moe_route")
        logits, expert = ctx.saved_tensors
        return route_backward(_gradient(dweight), logits, Routing(expert, None, None, None, None, ctx.params)), \
            None, None, None


def moe_route(logits: torch.Tensor, top_k: int, **options) -> Routing:
    """``route`` with gradients: those of the result's ``weight`` reach the logits [tokens, experts] (the choice
    of experts itself has none, and neither has the bias).  Options as for ``route``."""
    _refuse_captured_gradients("moe_route", logits)
    if not logits.requires_grad:
        return route(logits, top_k, **options)
    kept = []
    weight, expert, group_offsets, row_index, slot_row = _Route.apply(logits, top_k, options, kept)
    return Routing(expert, weight, group_offsets, row_index, slot_row, kept[0])


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, weight, slot_row, group_offsets, base):
        ctx.save_for_backward(rows, weight, slot_row, group_offsets)
        return combine(rows, slot_row, weight, base)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        _refuse_capture("moe_combine")
        rows, weight, slot_row, group_offsets = ctx.saved_tensors
        drows = dweight = None
        if ctx.needs_input_grad[0] or ctx.needs_input_grad[1]:
            drows, dweight = combine_backward(_gradient(dout), rows, slot_row, weight, group_offsets)
        return drows, dweight, None, None, dout if ctx.needs_input_grad[4] else None


def moe_combine(rows: torch.Tensor, routing: Routing, base: torch.Tensor | None = None) -> torch.Tensor:
    """out[t] = base[t] + sum_j routing.weight[t, j] * rows[routing.slot_row[t, j]] with gradients of rows (bf16 or
    f32, in the routing's order), of the weights and of base."""
    _refuse_captured_gradients("moe_combine", rows, routing.weight, base)
    return _Combine.apply(rows, routing.weight, routing.slot_row, routing.group_offsets, base)


@dataclass
class ExpertWeights:
    """One NVFP4 matrix [n, k] per expert, as ``grouped_gemm`` takes them: codes [experts, n, k/2], tiled scales,
    scales [experts]."""
    q: torch.Tensor
    sf: torch.Tensor
    g: torch.Tensor
    n: int


@torch.no_grad()
def expert_gemv(x: torch.Tensor, routing: Routing, up: ExpertWeights, down: ExpertWeights,
                base: torch.Tensor | None = None, activation=None) -> torch.Tensor:
    """The experts' forward pass of a few tokens x [tokens, hidden] bf16: each routed row through its expert's up
    matrix, ``activation`` (none by default; a function of the bf16 rows, each on its own), its down matrix, and
    the weighted sum per token on top of base.  x stays in bf16 (the products do not quantise it).  For inference:
    no gradients.  Of rows without an expert (routing.row_index -1) nothing is read."""
    h = grouped_gemv(routing.group_offsets, x, up.q, up.sf, up.g, up.n, routing.row_index, NVFP4_OUT_BF16)
    if activation is not None:
        h = activation(h)
    rows = grouped_gemv(routing.group_offsets, h, down.q, down.sf, down.g, down.n, None, NVFP4_OUT_F32)
    return combine(rows, routing.slot_row, routing.weight, base)


def expert_mlp(x: torch.Tensor, routing: Routing, up: ExpertWeights, down: ExpertWeights,
               gate: ExpertWeights | None = None, base: torch.Tensor | None = None) -> torch.Tensor:
    """``expert_gemv`` with the activation inside the products: silu(gate) * up, or max(up, 0)^2 without a gate.  The
    whole forward pass of a few tokens' experts, for inference: no gradients."""
    return _expert_mlp(x, routing, up, down, gate, base)
