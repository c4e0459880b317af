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

from .ops import (sl_embedding_fwd, sl_embedding_wgrad_accum, sl_linear_dgrad, sl_linear_dgrad_mxfp4, sl_linear_dgrad_mxfp8,
                  sl_linear_fwd, sl_linear_fwd_mxfp4, sl_linear_fwd_mxfp8, sl_linear_wgrad_accum, sl_linear_wgrad_accum_mxfp4,
                  sl_linear_wgrad_accum_mxfp8, sl_mxfp4_quantize, sl_mxfp8_quantize, sl_rmsnorm_bwd, sl_rmsnorm_fwd,
                  sl_rmsnorm_fwd_mxfp8, _raw_stream)


# A leaf has one gradient accumulator for all its living graphs, and it belongs to the stream on which it was made.  The functions below
# leave a weight's gradient in main_grad and return none, so a captured backward pass meets the accumulator's stream only at its
# end, where the engine joins that stream to the capture: if it is not the capture's, that ends the process.  So the functions
# note the stream on the accumulators that they meet, and refuse what a capture would do beside one noted on another: the
# linear functions a backward pass that comes to their weight's accumulator (torch.autograd.grad does not), the others the
# forward pass already, with the other leaves that they meet.  What they cannot know: an accumulator that other operators made, of a graph in which none of these functions has met the leaf, or
# on another stream than that of the first of these calls; and leaves behind an operator that comes before the call.

def _will_run(node):
    """Whether the backward pass under way runs an accumulator."""
    try:
        return torch._C._will_engine_execute_node(node)
    except RuntimeError:                  # torch.autograd.grad was asked for the leaf: it takes what flows there itself
        return False


def _refuse_foreign_accumulators(*leaves, in_backward=False):
    """Raises, while a graph is captured, for a leaf whose accumulator was noted on another stream."""
    for t in leaves:
        if t is not None and t.requires_grad and t.is_leaf and t.is_cuda:
            if not torch.cuda.is_current_stream_capturing():
                return
            stream = _raw_stream(t.device.index)
            node = torch.autograd.graph.get_gradient_edge(t).node
            if node.metadata.get("sl_stream", stream) != stream and (not in_backward or _will_run(node)):
                raise RuntimeError("a leaf's gradient accumulator belongs to another stream than the capture's and lives, held by a graph "
                                   "that was made there (drop its results before the capture) or by a hook on the accumulator: "
                                   "a backward pass cannot be captured beside it")


def _note_accumulators(out):
    """Notes the current stream on the accumulators next to the node that made ``out``."""
    fn = out.grad_fn
    if fn is not None and out.is_cuda:
        for node, _ in fn.next_functions:
            if node.__class__.__name__ == "AccumulateGrad":
                node.metadata.setdefault("sl_stream", _raw_stream(out.device.index))


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
        _refuse_foreign_accumulators(weight, in_backward=True)
        dy = grad_output.reshape(-1, grad_output.shape[-1]).contiguous()
        x2 = input.reshape(-1, input.shape[-1]).contiguous()
        dx = sl_linear_dgrad(dy, weight.detach())
        sl_linear_wgrad_accum(x2, dy, weight.main_grad)
        weight.grad_added_to_main_grad = True
        return dx.view(*input.shape), None


def linear_with_grad_accumulation(input: torch.Tensor, weight: torch.Tensor) -> torch.Tensor:
    y = LinearWithGradAccumulation.apply(input, weight)
    _note_accumulators(y)
    return y


def _check_copies(kind, copies, n_out, n_in, cols):
    """Checks (q_rows, s_rows, q_cols, s_cols) against the weight [n_out, n_in] whose copies in MXFP4 or MXFP8 they are; the
    columnwise pair is used, and may not be absent, only with ``cols``."""
    name = f"weight_{kind}"
    if len(copies) != 4:
        raise ValueError(f"{name} has {len(copies)} tensors, expected the four of sl_{kind}_quantize")
    if cols and (copies[2] is None or copies[3] is None):
        raise ValueError(f"the input gradient needs the weight's columnwise {kind.upper()} copy")
    out_b, in_b = (n_out + 31) // 32, (n_in + 31) // 32
    if kind == "mxfp4":
        shapes = ((n_out, 16 * in_b), (n_out, in_b), (n_in, 16 * out_b), (n_in, out_b))
    else:
        shapes = ((n_out, n_in), (n_out, in_b), (n_in, n_out), (n_in, out_b))
    for k, (t, shape) in enumerate(zip(copies, shapes[:4 if cols else 2])):
        if t is None or t.shape != shape:
            raise ValueError(f"{name}[{k}] of a weight [{n_out}, {n_in}] has shape {shape}, "
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
            _check_copies("mxfp4", weight_mxfp4, *weight.shape, ctx.needs_input_grad[0])
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
        _refuse_foreign_accumulators(weight, in_backward=True)
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
    y = LinearMXFP4WithGradAccumulation.apply(input, weight, seed, weight_mxfp4)
    _note_accumulators(y)
    return y


def _need_main_grad(weight, needed):
    if needed and not hasattr(weight, "main_grad"):
        raise ValueError("gradient accumulation fusion needs weight.main_grad (a grad_data view)")


class EmbeddingWithGradAccumulation(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ids, weight, vocab_start, scale):
        _need_main_grad(weight, ctx.needs_input_grad[1])
        ids = ids.contiguous()
        ctx.save_for_backward(ids, weight)
        ctx.at = vocab_start, scale
        return sl_embedding_fwd(ids, weight.detach(), vocab_start=vocab_start, scale=scale)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_output):
        ids, weight = ctx.saved_tensors
        sl_embedding_wgrad_accum(ids, grad_output.contiguous(), weight.main_grad, *ctx.at)
        weight.grad_added_to_main_grad = True
        return None, None, None, None


def embedding_with_grad_accumulation(ids: torch.Tensor, weight: torch.Tensor, vocab_start: int = 0, scale: float = 1.0) -> torch.Tensor:
    """Rows of the table shard ``weight`` [V, H] for ids of any shape, times ``scale``; zeros for ids of other ranks (outside
    vocab_start .. vocab_start + V - 1), so that the ranks' results add up.  Backward adds into weight.main_grad."""
    if torch.is_grad_enabled():
        _refuse_foreign_accumulators(weight)
    else:
        weight = weight.detach()
    y = EmbeddingWithGradAccumulation.apply(ids, weight, vocab_start, scale)
    _note_accumulators(y)
    return y


def _result(x, features):
    """A new result of ``features`` for each row of x, in x's shape from the start: what a Function returns as a view cannot be
    modified in place."""
    return torch.empty(*x.shape[:-1], features, dtype=torch.bfloat16, device=x.device)


def _rows(t):
    """t as contiguous rows of its last axis."""
    return None if t is None else t.reshape(-1, t.shape[-1]).contiguous()


def _norm_rows(x, weight, residual):
    """x and the residual as contiguous rows of the norm's width."""
    if weight.dim() != 1 or x.shape[-1] != weight.shape[0]:
        raise ValueError(f"input of {x.shape[-1]} features by a norm weight of shape {tuple(weight.shape)}")
    if residual is not None and residual.shape != x.shape:
        raise ValueError(f"residual has shape {tuple(residual.shape)}, the input {tuple(x.shape)}")
    return _rows(x), _rows(residual)


class RMSNormWithGradAccumulation(torch.autograd.Function):
    @staticmethod
    def forward(ctx, input, weight, residual, eps):
        _need_main_grad(weight, ctx.needs_input_grad[1])
        x2, r2 = _norm_rows(input, weight, residual)
        y, h = _result(input, input.shape[-1]), x2 if residual is None else _result(input, input.shape[-1])
        _, _, rstd = sl_rmsnorm_fwd(x2, weight.detach(), eps, residual=r2, y=_rows(y), h=None if residual is None else _rows(h))
        ctx.save_for_backward(h, weight, rstd)
        ctx.set_materialize_grads(False)
        ctx.shape = input.shape
        return y if residual is None else (y, h)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_y, grad_h=None):
        h, weight, rstd = ctx.saved_tensors
        return _norm_backward(ctx, grad_y, grad_h, h, weight, rstd) + (None,)


def _norm_backward(ctx, grad_y, grad_h, h, weight, rstd):
    """Gradients of input, weight (into main_grad) and residual."""
    if grad_y is None:
        return grad_h, None, grad_h if ctx.needs_input_grad[2] else None
    need_w = ctx.needs_input_grad[1]
    dx = sl_rmsnorm_bwd(_rows(grad_y), _rows(h), weight.detach(), rstd, weight.main_grad if need_w else None,
                        dresidual=_rows(grad_h)).view(ctx.shape)
    if need_w:
        weight.grad_added_to_main_grad = True
    return dx, None, dx if ctx.needs_input_grad[2] else None


def rmsnorm_with_grad_accumulation(input: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None,
                                   eps: float = 1e-5):
    """The root-mean-square norm of ``input`` over its last axis, or of h = input + residual: returns y, or (y, h), h being
    the residual stream that the next block adds to (out of place: backward reads h, and refuses one that was modified).  The
    weight's gradient goes to weight.main_grad."""
    if torch.is_grad_enabled():
        _refuse_foreign_accumulators(input, weight, residual)
    else:
        weight = weight.detach()
    out = RMSNormWithGradAccumulation.apply(input, weight, residual, eps)
    _note_accumulators(out if residual is None else out[0])
    return out


class NormLinearMXFP8WithGradAccumulation(torch.autograd.Function):
    """A norm and the all-MXFP8 linear step behind it.  The norm writes the step's input in MXFP8, along both axes at once, and
    in no other form; backward keeps its columnwise copy, the weight's, and h."""

    @classmethod
    def apply(cls, input, norm_weight, residual, weight, eps, weight_mxfp8):
        if not torch.is_grad_enabled():      # needs_input_grad tells of the tensors alone
            input, norm_weight, weight = input.detach(), norm_weight.detach(), weight.detach()
            residual = None if residual is None else residual.detach()
        return super().apply(input, norm_weight, residual, weight, eps, weight_mxfp8)

    @staticmethod
    def forward(ctx, input, norm_weight, residual, weight, eps, weight_mxfp8):
        need_x = any(ctx.needs_input_grad[:3])
        need_w = ctx.needs_input_grad[3]
        _need_main_grad(norm_weight, ctx.needs_input_grad[1])
        _need_main_grad(weight, need_w)
        if weight.dim() != 2 or input.shape[-1] != weight.shape[1]:
            raise ValueError(f"input of {input.shape[-1]} features by a weight of shape {tuple(weight.shape)}")
        x2, r2 = _norm_rows(input, norm_weight, residual)
        n_out, n_in = weight.shape
        T = x2.shape[0]
        if (need_w and T % 128) or (need_x and n_out % 128) or n_in % 32:
            raise ValueError(f"MXFP8 products of {T} tokens by a weight {(n_out, n_in)}: the contracted extents of the gradients "
                             "are multiples of 128, the input's of 32")
        if weight_mxfp8 is None:
            weight_mxfp8 = sl_mxfp8_quantize(weight.detach(), cols=need_x)
        else:
            _check_copies("mxfp8", weight_mxfp8, n_out, n_in, need_x)
        wr, wrs, wc, wcs = weight_mxfp8
        y, h = _result(input, n_out), x2 if residual is None else _result(input, n_in)
        xr, xrs, xc, xcs, _, rstd = sl_rmsnorm_fwd_mxfp8(x2, norm_weight.detach(), eps, residual=r2, cols=need_w,
                                                         h=None if residual is None else _rows(h))
        sl_linear_fwd_mxfp8(xr, xrs, wr, wrs, _rows(y))
        ctx.save_for_backward(h, norm_weight, rstd, weight, xc, xcs, wc, wcs)
        ctx.set_materialize_grads(False)
        ctx.shape = input.shape
        return y if residual is None else (y, h)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_y, grad_h=None):
        h, norm_weight, rstd, weight, xc, xcs, wc, wcs = ctx.saved_tensors
        grad_n = None
        if grad_y is not None:
            need_x, need_w = any(ctx.needs_input_grad[:3]), ctx.needs_input_grad[3]
            dy = grad_y.reshape(-1, grad_y.shape[-1]).contiguous()
            dr, drs, dc, dcs = sl_mxfp8_quantize(dy, rows=need_x, cols=need_w)
            if need_x:
                grad_n = sl_linear_dgrad_mxfp8(dr, drs, wc, wcs)
            if need_w:
                sl_linear_wgrad_accum_mxfp8(dc, dcs, xc, xcs, weight.main_grad)
                weight.grad_added_to_main_grad = True
        return _norm_backward(ctx, grad_n, grad_h, h, norm_weight, rstd) + (None, None, None)


def norm_linear_mxfp8_with_grad_accumulation(input: torch.Tensor, norm_weight: torch.Tensor, weight: torch.Tensor,
                                             residual: torch.Tensor | None = None, eps: float = 1e-5, weight_mxfp8=None):
    """Y = norm(input + residual) . weight^T with every product of the step on MXFP8 operands: returns Y, or (Y, h) with a
    residual, h = input + residual (which backward reads again).  Both weights' gradients go to their main_grad.  ``weight_mxfp8`` is
    sl_mxfp8_quantize(weight), made once and passed to every micro-batch; without it the weight is quantised in each call."""
    if torch.is_grad_enabled():
        _refuse_foreign_accumulators(input, norm_weight, residual, weight)
    out = NormLinearMXFP8WithGradAccumulation.apply(input, norm_weight, residual, weight, eps, weight_mxfp8)
    _note_accumulators(out if residual is None else out[0])
    return out
