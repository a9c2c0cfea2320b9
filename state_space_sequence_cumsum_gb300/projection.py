"""The projections around the scan in 8 bits (same names as ``include/ssd.h``):
matrices of 8-bit floats with a scale for each block of 128, their products, and
a layer's projection with its gradients.

An 8-bit matrix is two tensors: values [rows, cols] (float8_e4m3fn or
float8_e5m2, rows on 16-byte boundaries, which a padded row stride gives) and f32
scales, [rows, ceil(cols / 128)] by row or [ceil(rows / 128), ceil(cols / 128)]
by tile, of any strides.
"""
from __future__ import annotations

import torch

from ._autograd import first_order
from .layer import _call
from .ssd import Workspace

__all__ = ["ssd_block_quantize", "ssd_block_matmul", "ssd_projection", "ssd_projection_bwd", "ProjectionFunction"]

_FP8 = (torch.float8_e4m3fn, torch.float8_e5m2)


def ssd_block_quantize(x, tile=False, fp8=torch.float8_e4m3fn, want_q=True, want_t=False, stream=None):
    """x [rows, cols] bf16 or f32 (rows evenly spaced) in 8 bits, with a
    power-of-two scale for each 128 of a row or, with ``tile``, for each 128 x
    128: the least that brings the block's largest magnitude into the type.
    Returns (values, scales, values of the transpose, its scales); the first two
    are None without want_q, the others without want_t.  The transpose is
    quantised along its own rows; of tiles it holds the same values."""
    if fp8 not in _FP8:
        raise TypeError(f"fp8 must be float8_e4m3fn or float8_e5m2, got {fp8}")
    return _call("block_quantize", stream, x, tile, fp8 == torch.float8_e5m2, want_q, want_t)


def ssd_block_matmul(a, a_scale, b, b_scale, out_dtype=torch.bfloat16, out=None, stream=None):
    """a [m, k] times the transpose of b [n, k], two 8-bit matrices; out [m, n]
    bf16 or f32, summed in f32."""
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"out_dtype must be bfloat16 or float32, got {out_dtype}")
    return _call("block_matmul", stream, a, a_scale, b, b_scale, out_dtype == torch.bfloat16, out)


def ssd_projection(x, weight, weight_scale, return_kept=False, y=None, workspace: Workspace | None = None,
                   stream=None):
    """x [..., inputs] bf16 or f32 times the transpose of an 8-bit weight
    [outputs, inputs], x in 8 bits by token and 128 inputs.  Returns (y [...,
    outputs] in x's dtype, and with return_kept x's transpose [inputs, tokens] in
    8 bits and its scales, from which ssd_projection_bwd forms the weight's
    gradient, else None, None)."""
    return _call("projection", stream, x, weight, weight_scale, return_kept, y, workspace)


def ssd_projection_bwd(dy, weight_t=None, weight_t_scale=None, x_t=None, x_t_scale=None,
                       workspace: Workspace | None = None, stream=None):
    """Gradients of ssd_projection for dy [..., outputs]: dx (dy's dtype) from
    the weight's transpose [inputs, outputs] in 8 bits, dweight [outputs, inputs]
    f32 from what the forward kept.  dy is quantised along the outputs for the
    one and along the tokens for the other.  Returns a dict; what is not given
    has no gradient formed from it (None)."""
    return dict(zip(("dx", "dweight"),
                    _call("projection_bwd", stream, dy, weight_t, weight_t_scale, x_t, x_t_scale, workspace)))


class ProjectionFunction(torch.autograd.Function):
    """torch.autograd binding: apply(x, weight) -> x times the transpose of
    weight [outputs, inputs] (f32 or bf16, as the optimiser holds it), which is
    quantised by tiles for this call.  Kept for the backward: one byte for each
    element of x and of the weight."""

    @staticmethod
    def forward(ctx, x, weight):
        need_x, need_w = ctx.needs_input_grad
        q, scale, q_t, scale_t = ssd_block_quantize(weight, tile=True, want_t=need_x)
        y, x_t, x_t_scale = ssd_projection(x, q, scale, return_kept=need_w)
        ctx.save_for_backward(q_t, scale_t, x_t, x_t_scale)
        ctx.weight_dtype = weight.dtype
        return y

    @staticmethod
    @first_order
    def backward(ctx, dy):
        g = ssd_projection_bwd(dy.contiguous(), *ctx.saved_tensors)
        dw = g["dweight"]
        return g["dx"], None if dw is None else dw.to(ctx.weight_dtype)
