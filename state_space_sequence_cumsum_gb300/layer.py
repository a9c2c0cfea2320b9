"""Tensor-level binding of the layer operators around the scan (same names as
``include/ssd.h``): the short causal convolution, the selective scan and the
norms between blocks, with their gradients and single-token forms.

As in ``ssd.py``, PyTorch only allocates outputs and workspace and supplies
the stream; every arithmetic step runs in the library's kernels.  Checks and
allocations are compiled (``csrc/binding.cpp``).  Per-token
inputs (x, u, dt, z, B, C, dy) may be slices of wider projection outputs: the
last dimension contiguous, all other dimensions one even run of rows.
"""
from __future__ import annotations

import torch

from . import _lib
from ._autograd import first_order
from .ssd import Workspace

__all__ = ["ssd_causal_conv", "ssd_causal_conv_bwd", "ssd_causal_conv_step", "ssd_selective_scan",
           "ssd_selective_scan_bwd", "ssd_selective_scan_step", "ssd_selective_scan_chunk",
           "ssd_block_norm", "ssd_block_norm_bwd", "CausalConvFunction", "SelectiveScanFunction",
           "BlockNormFunction"]


def _call(name, stream, *args):
    """Calls the native binding on ``stream`` (None: the current one): outputs,
    and a workspace that is not given, come from that stream's pool; inputs and
    a given Workspace's buffer are kept for it.  One Workspace serves calls that
    are ordered, on one stream or by events between several."""
    f = getattr(_lib.native(), name)
    if stream is None:
        return f(*args)
    with torch.cuda.stream(stream):
        out = f(*args)
    for t in args:
        if isinstance(t, torch.Tensor):
            t.record_stream(stream)
    return out


def _given(grad, like=None):
    """An output's gradient, contiguous; where that output was not used, zeros
    like ``like`` or None."""
    if grad is not None:
        return grad.contiguous()
    return None if like is None else torch.zeros_like(like, memory_format=torch.contiguous_format)


# ------------------------------------------------------------- convolution

def _silu(activation):
    if activation not in (None, "silu", "swish"):
        raise ValueError("activation must be None or 'silu'")
    return activation is not None


def ssd_causal_conv(x, weight, bias=None, activation="silu", initial_state=None,
                    return_final_state=False, y=None, final_state=None, stream=None):
    """Causal depthwise convolution over the last ``width`` tokens, then SiLU
    (``activation=None``: none).  x [batch, seqlen, dim] bf16 or f32, weight
    [dim, width] and bias [dim] f32, initial_state [batch, width - 1, dim] in
    x's dtype: the tokens before x, oldest first (None: zeros).  Returns (y,
    the last width - 1 tokens or None)."""
    return _call("causal_conv", stream, x, weight, bias, _silu(activation), initial_state,
                 return_final_state, y, final_state)


def ssd_causal_conv_bwd(x, weight, dy, bias=None, activation="silu", initial_state=None,
                        dfinal=None, want_dinit=True, workspace: Workspace | None = None,
                        stream=None):
    """Gradients of ssd_causal_conv for dy (and dfinal, of the final state).
    Returns a dict with dx, dweight, dbias (None without bias) and dinit (None
    unless want_dinit)."""
    g = _call("causal_conv_bwd", stream, x, weight, dy, bias, _silu(activation), initial_state,
              dfinal, want_dinit, workspace)
    return dict(zip(("dx", "dweight", "dbias", "dinit"), g))


def ssd_causal_conv_step(x, weight, state, bias=None, activation="silu", state_out=None, y=None,
                         stream=None):
    """One token of ssd_causal_conv: x [batch, dim], state [batch, width - 1,
    dim] the tokens before it.  The state with x appended goes to
    ``state_out`` (default: ``state`` itself).  Returns (y, state_out)."""
    return _call("causal_conv_step", stream, x, weight, state, bias, _silu(activation), state_out, y)


class CausalConvFunction(torch.autograd.Function):
    """torch.autograd binding of ssd_causal_conv: apply(x, weight, bias,
    initial_state, activation) -> (y, final state)."""

    @staticmethod
    def forward(ctx, x, weight, bias=None, initial_state=None, activation="silu"):
        y, final = ssd_causal_conv(x, weight, bias, activation, initial_state,
                                   return_final_state=True)
        ctx.save_for_backward(x, weight, bias, initial_state)
        ctx.activation = activation
        ctx.set_materialize_grads(False)
        return y, final

    @staticmethod
    @first_order
    def backward(ctx, dy, dfinal):
        x, weight, bias, init = ctx.saved_tensors
        g = ssd_causal_conv_bwd(x, weight, _given(dy, x), bias, ctx.activation, init, _given(dfinal),
                                want_dinit=init is not None and ctx.needs_input_grad[3])
        return g["dx"], g["dweight"], g["dbias"], g["dinit"], None


# ---------------------------------------------------------- selective scan

def ssd_selective_scan_chunk() -> int:
    """Tokens between the states ssd_selective_scan keeps as chunk_states."""
    return int(_lib.load().ssd_selective_scan_chunk())


def ssd_selective_scan(u, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus=True,
                       initial_state=None, return_final_state=True, return_chunk_states=False,
                       y=None, final_state=None, chunk_states=None,
                       workspace: Workspace | None = None, stream=None):
    """Selective scan of a prompt: u, dt, z [batch, seqlen, dim] and B, C
    [batch, seqlen, (ngroups,) dstate] bf16 or f32, A [dim, dstate], D and
    dt_bias [dim], initial_state [batch, dim, dstate] f32.  Returns (y, final
    state or None, chunk states or None); the chunk states [batch, chunks,
    dim, dstate] are what ssd_selective_scan_bwd starts from.  final_state may
    be initial_state (in place)."""
    return _call("selective_scan", stream, u, dt, A, B, C, D, z, dt_bias, dt_softplus, initial_state,
                 return_final_state, return_chunk_states, y, final_state, chunk_states, workspace)


def ssd_selective_scan_bwd(u, dt, A, B, C, D, dy, z=None, dt_bias=None, dt_softplus=True,
                           initial_state=None, dfinal=None, chunk_states=None, want_dinit=True,
                           workspace: Workspace | None = None, stream=None):
    """Gradients of ssd_selective_scan for dy (and dfinal, of the final state,
    f32).  chunk_states: the forward's (None: recomputed).  Returns a dict with
    du, ddt, dA, dB, dC, dD, dz, ddt_bias and dinit (None where the input is
    absent; dinit None unless want_dinit)."""
    g = _call("selective_scan_bwd", stream, u, dt, A, B, C, D, dy, z, dt_bias, dt_softplus,
              initial_state, dfinal, chunk_states, want_dinit, workspace)
    return dict(zip(("du", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dinit"), g))


def ssd_selective_scan_step(u, dt, A, B, C, D, state, z=None, dt_bias=None, dt_softplus=True,
                            state_out=None, y=None, stream=None):
    """One token of ssd_selective_scan: u, dt, z [batch, dim], B, C [batch,
    (ngroups,) dstate], state [batch, dim, dstate] f32.  The updated state
    goes to ``state_out`` (default: ``state`` itself).  Returns (y, state_out)."""
    return _call("selective_scan_step", stream, u, dt, A, B, C, D, state, z, dt_bias, dt_softplus,
                 state_out, y)


class SelectiveScanFunction(torch.autograd.Function):
    """torch.autograd binding of ssd_selective_scan: apply(u, dt, A, B, C, D,
    z, dt_bias, initial_state, dt_softplus) -> (y, final state).  The forward
    keeps the chunk states its backward starts from, in f32: dstate / 8 times
    the bytes of a bf16 u.  Without a gradient to come it keeps none."""

    @classmethod
    def apply(cls, *args):
        if torch.is_grad_enabled() and any(isinstance(t, torch.Tensor) and t.requires_grad for t in args):
            return super().apply(*args)
        return cls._forward(*args)[:2]

    @staticmethod
    def _forward(u, dt, A, B, C, D=None, z=None, dt_bias=None, initial_state=None, dt_softplus=True, *,
                 keep=False):
        return ssd_selective_scan(u, dt, A, B, C, D, z, dt_bias, dt_softplus, initial_state, return_chunk_states=keep)

    @staticmethod
    def forward(ctx, u, dt, A, B, C, D=None, z=None, dt_bias=None, initial_state=None,
                dt_softplus=True):
        y, final, kept = SelectiveScanFunction._forward(u, dt, A, B, C, D, z, dt_bias, initial_state, dt_softplus,
                                                        keep=True)
        ctx.save_for_backward(u, dt, A, B, C, D, z, dt_bias, initial_state, kept)
        ctx.dt_softplus = dt_softplus
        ctx.set_materialize_grads(False)
        return y, final

    @staticmethod
    @first_order
    def backward(ctx, dy, dfinal):
        u, dt, A, B, C, D, z, dt_bias, init, kept = ctx.saved_tensors
        g = ssd_selective_scan_bwd(u, dt, A, B, C, D, _given(dy, u), z, dt_bias, ctx.dt_softplus, init,
                                   _given(dfinal), kept, want_dinit=init is not None and ctx.needs_input_grad[8])
        return (g["du"], g["ddt"], g["dA"], g["dB"], g["dC"], g["dD"], g["dz"], g["ddt_bias"],
                g["dinit"], None)


# -------------------------------------------------------------- block norm

def ssd_block_norm(y, residual, weight, post_weight=None, gate=None, scale=1.0, eps=1e-5, out=None,
                   residual_out=None, residual_dtype=None, stream=None):
    """What stands between two blocks: p = rmsnorm(y) * post_weight (or y),
    residual_out = residual + scale * gate * p, out = rmsnorm(residual_out) *
    weight.  y [..., dim] bf16 or f32, residual in y's dtype or f32 (None:
    zeros, and residual_dtype, y's or f32, is residual_out's), weights [dim]
    and gate [..., dim] f32 with one row for all tokens, for equal runs of
    them (one per sequence) or for each.  Returns (out, residual_out);
    residual_out may be residual (in place).  A residual_dtype other than that
    of a given residual or residual_out is refused."""
    if residual_dtype not in (None, torch.float32, y.dtype):
        raise TypeError(f"the residual must be {y.dtype} or float32, got {residual_dtype}")
    for name, t in (("residual", residual), ("residual_out", residual_out)):
        if residual_dtype is not None and t is not None and t.dtype != residual_dtype:
            raise TypeError(f"{name} is {t.dtype}, residual_dtype {residual_dtype}")
    return _call("block_norm", stream, y, residual, weight, post_weight, gate, scale, eps, out,
                 residual_out, residual_dtype == torch.float32)


def ssd_block_norm_bwd(y, residual_out, weight, dout, dresidual_out=None, post_weight=None,
                       gate=None, scale=1.0, eps=1e-5, workspace: Workspace | None = None,
                       stream=None):
    """Gradients of ssd_block_norm from its y and residual_out, for dout and
    dresidual_out (None: zero).  Returns a dict with dy, dresidual, dweight,
    dpost_weight and dgate (None where the input is absent)."""
    g = _call("block_norm_bwd", stream, y, residual_out, weight, dout, dresidual_out, post_weight,
              gate, scale, eps, workspace)
    return dict(zip(("dy", "dresidual", "dweight", "dpost_weight", "dgate"), g))


class BlockNormFunction(torch.autograd.Function):
    """torch.autograd binding of ssd_block_norm: apply(y, residual, weight,
    post_weight, gate, scale, eps) -> (out, residual_out)."""

    @staticmethod
    def forward(ctx, y, residual, weight, post_weight=None, gate=None, scale=1.0, eps=1e-5):
        out, res = ssd_block_norm(y, residual, weight, post_weight, gate, scale, eps)
        ctx.save_for_backward(y, res, weight, post_weight, gate)
        ctx.scalars = (scale, eps)
        ctx.has_residual = residual is not None
        ctx.set_materialize_grads(False)
        return out, res

    @staticmethod
    @first_order
    def backward(ctx, dout, dres):
        y, res, weight, post_weight, gate = ctx.saved_tensors
        g = ssd_block_norm_bwd(y, res, weight, _given(dout, y), _given(dres), post_weight, gate, *ctx.scalars)
        return (g["dy"], g["dresidual"] if ctx.has_residual else None, g["dweight"],
                g["dpost_weight"], g["dgate"], None, None)
