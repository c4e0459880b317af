"""Autograd function of the linear step with gradient-accumulation fusion.

llm-infra-atlas "01 · ColumnParallelLinear / RowParallelLinear and the core autograd",
section 4: forward saves (input, weight) and computes Y = X.W^T; backward computes the input
gradient dY.W, then the weight gradient straight into the fp32 weight.main_grad, returns no
weight gradient and marks weight.grad_added_to_main_grad.  Communication (sequence-parallel
all-gather, dgrad all-reduce / reduce-scatter) is outside this single-GPU step.
"""
from __future__ import annotations

import torch

from torch.autograd.function import once_differentiable

from .ops import (sl_linear_dgrad, sl_linear_dgrad_mxfp4, sl_linear_fwd, sl_linear_fwd_mxfp4, sl_linear_wgrad_accum,
                  sl_linear_wgrad_accum_mxfp4, sl_mxfp4_quantize)


class LinearWithGradAccumulation(torch.autograd.Function):
    @staticmethod
    def forward(ctx, input: torch.Tensor, weight: torch.Tensor):
        if not hasattr(weight, "main_grad"):
            raise ValueError("gradient accumulation fusion needs weight.main_grad (a grad_data view)")
        x2 = input.reshape(-1, input.shape[-1])
        y = sl_linear_fwd(x2.contiguous(), weight.detach())
        ctx.save_for_backward(input, weight)
        return y.view(*input.shape[:-1], weight.shape[0])

    @staticmethod
    def backward(ctx, grad_output: torch.Tensor):
        input, weight = ctx.saved_tensors
        dy = grad_output.reshape(-1, grad_output.shape[-1]).contiguous()
        x2 = input.reshape(-1, input.shape[-1]).contiguous()
        dx = sl_linear_dgrad(dy, weight.detach())
        sl_linear_wgrad_accum(x2, dy, weight.main_grad)
        weight.grad_added_to_main_grad = True
        return dx.view(*input.shape), None


def linear_with_grad_accumulation(input: torch.Tensor, weight: torch.Tensor) -> torch.Tensor:
    return LinearWithGradAccumulation.apply(input, weight)


def _check_copies(copies, n_out, n_in, cols):
    """Checks (q_rows, s_rows, q_cols, s_cols) against the weight [n_out, n_in] whose copies they are; the
    columnwise pair is used, and may not be absent, only with ``cols``."""
    if len(copies) != 4:
        raise ValueError(f"weight_mxfp4 has {len(copies)} tensors, expected the four of sl_mxfp4_quantize")
    if cols and (copies[2] is None or copies[3] is None):
        raise ValueError("the input gradient needs the weight's columnwise MXFP4 copy")
    out_b, in_b = (n_out + 31) // 32, (n_in + 31) // 32
    shapes = ((n_out, 16 * in_b), (n_out, in_b), (n_in, 16 * out_b), (n_in, out_b))
    for k, (t, shape) in enumerate(zip(copies, shapes[:4 if cols else 2])):
        if t is None or t.shape != shape:
            raise ValueError(f"weight_mxfp4[{k}] of a weight [{n_out}, {n_in}] has shape {shape}, "
                             f"got {None if t is None else tuple(t.shape)}")


class LinearMXFP4WithGradAccumulation(torch.autograd.Function):
    """The linear step with every product on MXFP4 operands: X, W and dY are cast inside the step, each
    along the axis its product contracts.  What is kept for backward is X's columnwise copy (0.53 bytes an
    element) and W's; without gradients neither is made."""

    @classmethod
    def apply(cls, input, weight, seed=None, weight_mxfp4=None):
        if not torch.is_grad_enabled():      # needs_input_grad tells of the tensors alone
            input, weight = input.detach(), weight.detach()
        return super().apply(input, weight, seed, weight_mxfp4)

    @staticmethod
    def forward(ctx, input, weight, seed, weight_mxfp4):
        if ctx.needs_input_grad[1] and not hasattr(weight, "main_grad"):
            raise ValueError("gradient accumulation fusion needs weight.main_grad (a grad_data view)")
        if weight.dim() != 2 or input.shape[-1] != weight.shape[1]:
            raise ValueError(f"input of {input.shape[-1]} features by a weight of shape {tuple(weight.shape)}")
        if weight_mxfp4 is not None:
            _check_copies(weight_mxfp4, *weight.shape, ctx.needs_input_grad[0])
        x2 = input.reshape(-1, input.shape[-1]).contiguous()
        xr, xrs, xc, xcs = sl_mxfp4_quantize(x2, cols=ctx.needs_input_grad[1])
        if weight_mxfp4 is None:
            weight_mxfp4 = sl_mxfp4_quantize(weight.detach(), cols=ctx.needs_input_grad[0])
        wr, wrs, wc, wcs = weight_mxfp4
        y = sl_linear_fwd_mxfp4(xr, xrs, wr, wrs)
        ctx.save_for_backward(weight, xc, xcs, wc, wcs)
        ctx.seed, ctx.shape = seed, input.shape
        return y.view(*input.shape[:-1], weight.shape[0])

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_output):
        weight, xc, xcs, wc, wcs = ctx.saved_tensors
        dy = grad_output.reshape(-1, grad_output.shape[-1]).contiguous()
        need_x, need_w = ctx.needs_input_grad[:2]
        dr, drs, dc, dcs = sl_mxfp4_quantize(dy, rows=need_x, cols=need_w, seed=ctx.seed)
        dx = sl_linear_dgrad_mxfp4(dr, drs, wc, wcs).view(ctx.shape) if need_x else None
        if need_w:
            sl_linear_wgrad_accum_mxfp4(dc, dcs, xc, xcs, weight.main_grad)
            weight.grad_added_to_main_grad = True
        return dx, None, None, None


def linear_mxfp4_with_grad_accumulation(input: torch.Tensor, weight: torch.Tensor, seed=None,
                                        weight_mxfp4=None) -> torch.Tensor:
    """linear_with_grad_accumulation with all three products in MXFP4.  ``seed`` (see sl_mxfp4_quantize)
    rounds dY stochastically, which keeps the gradients unbiased; a training loop gives every call its
    own.  ``weight_mxfp4`` is sl_mxfp4_quantize(weight), made once and passed to every micro-batch that
    uses the same weight; without it the weight is cast in each call."""
    return LinearMXFP4WithGradAccumulation.apply(input, weight, seed, weight_mxfp4)
