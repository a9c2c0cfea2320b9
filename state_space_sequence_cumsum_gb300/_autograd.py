"""What the autograd bindings of the library's operators share."""
from __future__ import annotations

import functools

import torch


class _NoSecondOrder(torch.autograd.Function):
    """The first n tensors as they are, behind a node whose backward raises."""

    @staticmethod
    def forward(ctx, where, n, *tensors):
        ctx.where = where
        return tuple(None if t is None else t.view_as(t) for t in tensors[:n])

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError(f"{ctx.where} has no second-order gradients: its backward cannot be differentiated")


def first_order(backward):
    """Decorates the backward of an autograd function that runs in the
    library's kernels.  Its results are constants to autograd, so with
    create_graph=True a derivative through them would lose their share without
    an error; it raises instead.  (once_differentiable lets that pass where
    the incoming gradients are constants, as those of a plain sum are.)"""
    @functools.wraps(backward)
    def wrapper(ctx, *grads):
        with torch.no_grad():
            out = backward(ctx, *grads)
        if not torch.is_grad_enabled():
            return out
        at = [i for i, t in enumerate(out) if t is not None]
        marked = _NoSecondOrder.apply(type(ctx).__name__.removesuffix("Backward"), len(at), *[out[i] for i in at],
                                      *ctx.saved_tensors, *grads)
        out = list(out)
        for i, t in zip(at, marked):
            out[i] = t
        return tuple(out)
    return wrapper
