"""Tensor-level binding of the layer operators around the scan (same names as
``include/ssd.h``): the short causal convolution, the selective scan and the
norms between blocks, with their gradients and single-token forms.

As in ``ssd.py``, PyTorch only allocates outputs and workspace and supplies
the stream; every arithmetic step runs in the library's kernels.  Per-token
inputs (x, u, dt, z, B, C, dy) may be slices of wider projection outputs: the
last dimension contiguous, all other dimensions one even run of rows.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import _lib
from ._lib import check
from .ssd import Workspace, _dtype_code, _f32

__all__ = ["ssd_causal_conv", "ssd_causal_conv_bwd", "ssd_causal_conv_step", "ssd_selective_scan",
           "ssd_selective_scan_bwd", "ssd_selective_scan_step", "ssd_selective_scan_chunk",
           "ssd_block_norm", "ssd_block_norm_bwd", "CausalConvFunction", "SelectiveScanFunction",
           "BlockNormFunction"]


def _addr(t):
    return None if t is None else t.data_ptr()


def _row(t, name):
    """Elements between consecutive rows of t, whose rows are evenly spaced."""
    shape, stride = t.shape, t.stride()
    n = shape[-1]
    if stride[-1] != 1 and n > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    if t.numel() == 0:
        return n
    row, step = None, None
    for size, st in zip(reversed(shape[:-1]), reversed(stride[:-1])):
        if size == 1:
            continue
        if step is None:
            row = st
        elif st != step:
            raise ValueError(f"{name}: rows must be evenly spaced")
        step = st * size
    if row is None:
        return n
    if row < n:
        raise ValueError(f"{name}: rows overlap")
    return row


def _flat_groups(t, lead, name):
    """B or C with its [groups, dstate] as one dimension, and its groups."""
    if t.dim() == lead + 2:
        G = t.shape[-2]
        if t.shape[-1] > 1 and t.stride(-1) != 1 or G > 1 and t.stride(-2) != t.shape[-1]:
            raise ValueError(f"{name}: groups and states must be contiguous")
        return t.flatten(-2), G
    if t.dim() != lead + 1:
        raise ValueError(f"{name} must be [..., dstate] or [..., ngroups, dstate]")
    return t, 1


def _same(t, name, shape, dtype, device, contiguous=False):
    """Checks an optional tensor's shape, type and device."""
    if t is None:
        return None
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


class _On:
    """The call's device and stream: outputs and workspace are allocated on
    the stream the kernels run on, and inputs are kept for it."""

    def __init__(self, t, stream, inputs):
        if not t.is_cuda:
            raise ValueError("layer operators take CUDA tensors")
        self.stack = None
        index = t.device.index
        if torch.cuda.current_device() != index:
            self.stack = contextlib.ExitStack()
            self.stack.enter_context(torch.cuda.device(index))
        if stream is None:
            self.stream = torch.cuda.current_stream().cuda_stream
        else:
            self.stream = stream.cuda_stream
            if stream != torch.cuda.current_stream():
                self.stack = self.stack or contextlib.ExitStack()
                self.stack.enter_context(torch.cuda.stream(stream))
                for i in inputs:
                    if i is not None:
                        i.record_stream(stream)

    def __enter__(self):
        return self.stream

    def __exit__(self, *exc):
        if self.stack is not None:
            self.stack.close()
        return False


def _workspace(nbytes, workspace, device):
    """(address, size) of a workspace; the tensor is returned to be kept alive."""
    if nbytes == 0:
        return None, 0, None
    buf = workspace.get(nbytes, device) if workspace is not None else \
        torch.empty(nbytes, dtype=torch.uint8, device=device)
    return buf.data_ptr(), buf.numel(), buf


# ------------------------------------------------------------- convolution

def _activation(activation):
    if activation not in (None, "silu", "swish"):
        raise ValueError("activation must be None or 'silu'")
    return int(activation is not None)


def _conv_args(x, weight, bias, lead):
    code = _dtype_code(x)
    if x.dim() != lead + 1:
        raise ValueError("x must be [batch, seqlen, dim]" if lead == 2 else "x must be [batch, dim]")
    if weight.dim() != 2 or weight.shape[0] != x.shape[-1]:
        raise ValueError("weight must be [dim, width]")
    dev, dim, width = x.device, x.shape[-1], weight.shape[1]
    _same(weight, "weight", (dim, width), torch.float32, dev, True)
    _same(bias, "bias", (dim,), torch.float32, dev, True)
    seqlen = x.shape[1] if lead == 2 else 1
    return code, _lib.ssd_conv_dims_t(x.shape[0], seqlen, dim, width), (x.shape[0], max(width - 1, 0), dim)


def ssd_causal_conv(x, weight, bias=None, activation="silu", initial_state=None,
                    return_final_state=False, y=None, final_state=None, stream=None):
    """Causal depthwise convolution over the last ``width`` tokens, then SiLU
    (``activation=None``: none).  x [batch, seqlen, dim] bf16 or f32, weight
    [dim, width] and bias [dim] f32, initial_state [batch, width - 1, dim] in
    x's dtype: the tokens before x, oldest first (None: zeros).  Returns (y,
    the last width - 1 tokens or None)."""
    silu = _activation(activation)
    code, d, st_shape = _conv_args(x, weight, bias, 2)
    row = _row(x, "x")
    _same(initial_state, "initial_state", st_shape, x.dtype, x.device, True)
    with _On(x, stream, (x, weight, bias, initial_state)) as s:
        if y is None:
            y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        if final_state is None and return_final_state:
            final_state = torch.empty(st_shape, dtype=x.dtype, device=x.device)
        _same(y, "y", x.shape, x.dtype, x.device, True)
        _same(final_state, "final_state", st_shape, x.dtype, x.device, True)
        check(_lib.load().ssd_causal_conv(_addr(x), row, _addr(weight), _addr(bias),
                                          _addr(initial_state), _addr(y), _addr(final_state), d,
                                          silu, code, s), "ssd_causal_conv")
    return y, final_state


def ssd_causal_conv_bwd(x, weight, dy, bias=None, activation="silu", initial_state=None,
                        dfinal=None, want_dinit=True, workspace: Workspace | None = None,
                        stream=None):
    """Gradients of ssd_causal_conv for dy (and dfinal, of the final state).
    Returns a dict with dx, dweight, dbias (None without bias) and dinit (None
    unless want_dinit)."""
    silu = _activation(activation)
    code, d, st_shape = _conv_args(x, weight, bias, 2)
    _same(dy, "dy", x.shape, x.dtype, x.device)
    row, row_dy = _row(x, "x"), _row(dy, "dy")
    _same(initial_state, "initial_state", st_shape, x.dtype, x.device, True)
    _same(dfinal, "dfinal", st_shape, x.dtype, x.device, True)
    lib = _lib.load()
    with _On(x, stream, (x, weight, bias, initial_state, dy, dfinal)) as s:
        def new(shape, dtype):
            return torch.empty(shape, dtype=dtype, device=x.device)
        out = {"dx": new(x.shape, x.dtype), "dweight": new(weight.shape, torch.float32),
               "dbias": None if bias is None else new(bias.shape, torch.float32),
               "dinit": new(st_shape, x.dtype) if want_dinit else None}
        ws, size, _keep = _workspace(lib.ssd_causal_conv_bwd_workspace_size(d), workspace, x.device)
        check(lib.ssd_causal_conv_bwd(_addr(x), row, _addr(weight), _addr(bias),
                                      _addr(initial_state), _addr(dy), row_dy, _addr(dfinal),
                                      _addr(out["dx"]), _addr(out["dweight"]), _addr(out["dbias"]),
                                      _addr(out["dinit"]), d, silu, code, ws, size, s),
              "ssd_causal_conv_bwd")
    return out


def ssd_causal_conv_step(x, weight, state, bias=None, activation="silu", state_out=None, y=None,
                         stream=None):
    """One token of ssd_causal_conv: x [batch, dim], state [batch, width - 1,
    dim] the tokens before it.  The state with x appended goes to
    ``state_out`` (default: ``state`` itself).  Returns (y, state_out)."""
    silu = _activation(activation)
    code, d, st_shape = _conv_args(x, weight, bias, 1)
    row = _row(x, "x")
    state_out = state if state_out is None else state_out
    _same(state, "state", st_shape, x.dtype, x.device, True)
    _same(state_out, "state_out", st_shape, x.dtype, x.device, True)
    with _On(x, stream, (x, weight, bias, state, state_out)) as s:
        if y is None:
            y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        _same(y, "y", x.shape, x.dtype, x.device, True)
        check(_lib.load().ssd_causal_conv_step(_addr(x), row, _addr(weight), _addr(bias),
                                               _addr(state), _addr(state_out), _addr(y), d, silu,
                                               code, s), "ssd_causal_conv_step")
    return y, state_out


class CausalConvFunction(torch.autograd.Function):
    """torch.autograd binding of ssd_causal_conv: apply(x, weight, bias,
    initial_state, activation) -> (y, final state)."""

    @staticmethod
    def forward(ctx, x, weight, bias=None, initial_state=None, activation="silu"):
        y, final = ssd_causal_conv(x, weight, bias, activation, initial_state,
                                   return_final_state=True)
        ctx.save_for_backward(x, weight, bias, initial_state)
        ctx.activation = activation
        return y, final

    @staticmethod
    def backward(ctx, dy, dfinal):
        x, weight, bias, init = ctx.saved_tensors
        g = ssd_causal_conv_bwd(x, weight, dy.contiguous(), bias, ctx.activation, init,
                                dfinal.contiguous(), want_dinit=init is not None)
        return g["dx"], g["dweight"], g["dbias"], g["dinit"], None


# ---------------------------------------------------------- selective scan

def ssd_selective_scan_chunk() -> int:
    """Tokens between the states ssd_selective_scan keeps as chunk_states."""
    return int(_lib.load().ssd_selective_scan_chunk())


class _ScanArgs:
    """Checked shapes of a scan's inputs (lead: dimensions before dim)."""

    def __init__(self, u, dt, A, B, C, D, z, dt_bias, lead, dy=None):
        self.code = _dtype_code(u)
        if u.dim() != lead + 1:
            raise ValueError("u must be [batch, seqlen, dim]" if lead == 2 else "u must be [batch, dim]")
        dev, dim = u.device, u.shape[-1]
        if A.dim() != 2 or A.shape[0] != dim:
            raise ValueError("A must be [dim, dstate]")
        N = A.shape[1]
        self.bc_shape = B.shape
        _same(C, "C", B.shape, u.dtype, dev)
        self.B, G = _flat_groups(B, lead, "B")
        self.C, _ = _flat_groups(C, lead, "C")
        if dim % max(G, 1) != 0:
            raise ValueError("dim must be a multiple of the groups of B and C")
        _same(self.B, "B", u.shape[:-1] + (G * N,), u.dtype, dev)
        _same(dt, "dt", u.shape, u.dtype, dev)
        _same(z, "z", u.shape, u.dtype, dev)
        _same(dy, "dy", u.shape, u.dtype, dev)
        _same(A, "A", (dim, N), torch.float32, dev, True)
        _same(D, "D", (dim,), torch.float32, dev, True)
        _same(dt_bias, "dt_bias", (dim,), torch.float32, dev, True)
        self.dims = _lib.ssd_scan_dims_t(u.shape[0], u.shape[1] if lead == 2 else 1, dim, N, G)
        self.rows = _lib.ssd_scan_rows_t(_row(u, "u"), _row(dt, "dt"),
                                         dim if z is None else _row(z, "z"), _row(self.B, "B"),
                                         _row(self.C, "C"), dim if dy is None else _row(dy, "dy"))
        self.state_shape = (u.shape[0], dim, N)
        self.inputs = (u, dt, A, B, C, D, z, dt_bias, dy)


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
    a = _ScanArgs(u, dt, A, B, C, D, z, dt_bias, 2)
    lib = _lib.load()
    _same(initial_state, "initial_state", a.state_shape, torch.float32, u.device, True)
    nc = -(-u.shape[1] // lib.ssd_selective_scan_chunk())
    kept_shape = (u.shape[0], nc) + a.state_shape[1:]
    with _On(u, stream, a.inputs + (initial_state,)) as s:
        if y is None:
            y = torch.empty(u.shape, dtype=u.dtype, device=u.device)
        if final_state is None and return_final_state:
            final_state = torch.empty(a.state_shape, dtype=torch.float32, device=u.device)
        if chunk_states is None and return_chunk_states:
            chunk_states = torch.empty(kept_shape, dtype=torch.float32, device=u.device)
        _same(y, "y", u.shape, u.dtype, u.device, True)
        _same(final_state, "final_state", a.state_shape, torch.float32, u.device, True)
        _same(chunk_states, "chunk_states", kept_shape, torch.float32, u.device, True)
        ws, size, _keep = _workspace(lib.ssd_selective_scan_workspace_size(a.dims), workspace, u.device)
        check(lib.ssd_selective_scan(_addr(u), _addr(dt), _addr(A), _addr(a.B), _addr(a.C), _addr(D),
                                     _addr(z), _addr(dt_bias), _addr(initial_state), _addr(y),
                                     _addr(final_state), _addr(chunk_states), a.dims, a.rows,
                                     int(bool(dt_softplus)), a.code, ws, size, s),
              "ssd_selective_scan")
    return y, final_state, chunk_states


def ssd_selective_scan_bwd(u, dt, A, B, C, D, dy, z=None, dt_bias=None, dt_softplus=True,
                           initial_state=None, dfinal=None, chunk_states=None, want_dinit=True,
                           workspace: Workspace | None = None, stream=None):
    """Gradients of ssd_selective_scan for dy (and dfinal, of the final state,
    f32).  chunk_states: the forward's (None: recomputed).  Returns a dict with
    du, ddt, dA, dB, dC, dD, dz, ddt_bias and dinit (None where the input is
    absent; dinit None unless want_dinit)."""
    a = _ScanArgs(u, dt, A, B, C, D, z, dt_bias, 2, dy)
    lib = _lib.load()
    nc = -(-u.shape[1] // lib.ssd_selective_scan_chunk())
    dev, f32 = u.device, torch.float32
    _same(initial_state, "initial_state", a.state_shape, f32, dev, True)
    _same(dfinal, "dfinal", a.state_shape, f32, dev, True)
    _same(chunk_states, "chunk_states", (u.shape[0], nc) + a.state_shape[1:], f32, dev, True)
    with _On(u, stream, a.inputs + (initial_state, dfinal, chunk_states)) as s:
        def new(shape, dtype, want=True):
            return torch.empty(shape, dtype=dtype, device=dev) if want else None
        out = {"du": new(u.shape, u.dtype), "ddt": new(u.shape, u.dtype), "dA": new(A.shape, f32),
               "dB": new(a.bc_shape, u.dtype), "dC": new(a.bc_shape, u.dtype),
               "dD": new(A.shape[:1], f32, D is not None), "dz": new(u.shape, u.dtype, z is not None),
               "ddt_bias": new(A.shape[:1], f32, dt_bias is not None),
               "dinit": new(a.state_shape, f32, want_dinit)}
        nbytes = lib.ssd_selective_scan_bwd_workspace_size(a.dims, int(chunk_states is not None))
        ws, size, _keep = _workspace(nbytes, workspace, dev)
        check(lib.ssd_selective_scan_bwd(
            _addr(u), _addr(dt), _addr(A), _addr(a.B), _addr(a.C), _addr(D), _addr(z), _addr(dt_bias),
            _addr(initial_state), _addr(dy), _addr(dfinal), _addr(chunk_states), _addr(out["du"]),
            _addr(out["ddt"]), _addr(out["dA"]), _addr(out["dB"]), _addr(out["dC"]), _addr(out["dD"]),
            _addr(out["dz"]), _addr(out["ddt_bias"]), _addr(out["dinit"]), a.dims, a.rows,
            int(bool(dt_softplus)), a.code, ws, size, s), "ssd_selective_scan_bwd")
    return out


def ssd_selective_scan_step(u, dt, A, B, C, D, state, z=None, dt_bias=None, dt_softplus=True,
                            state_out=None, y=None, stream=None):
    """One token of ssd_selective_scan: u, dt, z [batch, dim], B, C [batch,
    (ngroups,) dstate], state [batch, dim, dstate] f32.  The updated state
    goes to ``state_out`` (default: ``state`` itself).  Returns (y, state_out)."""
    a = _ScanArgs(u, dt, A, B, C, D, z, dt_bias, 1)
    state_out = state if state_out is None else state_out
    _same(state, "state", a.state_shape, torch.float32, u.device, True)
    _same(state_out, "state_out", a.state_shape, torch.float32, u.device, True)
    with _On(u, stream, a.inputs + (state, state_out)) as s:
        if y is None:
            y = torch.empty(u.shape, dtype=u.dtype, device=u.device)
        _same(y, "y", u.shape, u.dtype, u.device, True)
        check(_lib.load().ssd_selective_scan_step(
            _addr(u), _addr(dt), _addr(A), _addr(a.B), _addr(a.C), _addr(D), _addr(z), _addr(dt_bias),
            _addr(state), _addr(state_out), _addr(y), a.dims, a.rows, int(bool(dt_softplus)), a.code,
            s), "ssd_selective_scan_step")
    return y, state_out


class SelectiveScanFunction(torch.autograd.Function):
    """torch.autograd binding of ssd_selective_scan: apply(u, dt, A, B, C, D,
    z, dt_bias, initial_state, dt_softplus) -> (y, final state).  The forward
    keeps the chunk states its backward starts from."""

    @staticmethod
    def forward(ctx, u, dt, A, B, C, D=None, z=None, dt_bias=None, initial_state=None,
                dt_softplus=True):
        y, final, kept = ssd_selective_scan(u, dt, A, B, C, D, z, dt_bias, dt_softplus,
                                            initial_state, return_chunk_states=True)
        ctx.save_for_backward(u, dt, A, B, C, D, z, dt_bias, initial_state, kept)
        ctx.dt_softplus = dt_softplus
        return y, final

    @staticmethod
    def backward(ctx, dy, dfinal):
        u, dt, A, B, C, D, z, dt_bias, init, kept = ctx.saved_tensors
        g = ssd_selective_scan_bwd(u, dt, A, B, C, D, dy.contiguous(), z, dt_bias, ctx.dt_softplus,
                                   init, dfinal.contiguous(), kept, want_dinit=init is not None)
        return (g["du"], g["ddt"], g["dA"], g["dB"], g["dC"], g["dD"], g["dz"], g["ddt_bias"],
                g["dinit"], None)


# -------------------------------------------------------------- block norm

def _norm_args(y, weight, post_weight, gate):
    code = _dtype_code(y)
    if y.dim() < 1:
        raise ValueError("y must be [..., dim]")
    dim, dev, f32 = y.shape[-1], y.device, torch.float32
    tokens = y.numel() // dim if dim else 0
    if not y.is_contiguous():
        raise ValueError("y must be contiguous")
    _same(weight, "weight", (dim,), f32, dev, True)
    _same(post_weight, "post_weight", (dim,), f32, dev, True)
    rows = 0
    if gate is not None:
        rows = gate.numel() // dim if dim else 0
        _same(gate, "gate", gate.shape[:-1] + (dim,), f32, dev, True)
        if rows < 1 or tokens % rows:
            raise ValueError("the tokens must be a multiple of the gate's rows")
    return code, tokens, dim, rows


def _residual_code(y, t):
    if t.dtype not in (y.dtype, torch.float32):
        raise TypeError(f"the residual must be {y.dtype} or float32, got {t.dtype}")
    return _dtype_code(t)


def ssd_block_norm(y, residual, weight, post_weight=None, gate=None, scale=1.0, eps=1e-5, out=None,
                   residual_out=None, residual_dtype=None, stream=None):
    """What stands between two blocks: p = rmsnorm(y) * post_weight (or y),
    residual_out = residual + scale * gate * p, out = rmsnorm(residual_out) *
    weight.  y [..., dim] bf16 or f32, residual in y's dtype or f32 (None:
    zeros, and residual_dtype says the type of residual_out), weights [dim] and
    gate [..., dim] f32 with one row for all tokens, for equal runs of them
    (one per sequence) or for each.  Returns (out, residual_out);
    residual_out may be residual (in place)."""
    code, tokens, dim, rows = _norm_args(y, weight, post_weight, gate)
    like = residual if residual is not None else residual_out
    rdt = like.dtype if like is not None else (residual_dtype or y.dtype)
    with _On(y, stream, (y, residual, weight, post_weight, gate)) as s:
        if out is None:
            out = torch.empty(y.shape, dtype=y.dtype, device=y.device)
        if residual_out is None:
            residual_out = torch.empty(y.shape, dtype=rdt, device=y.device)
        _same(out, "out", y.shape, y.dtype, y.device, True)
        _same(residual, "residual", y.shape, rdt, y.device, True)
        _same(residual_out, "residual_out", y.shape, rdt, y.device, True)
        check(_lib.load().ssd_block_norm(_addr(y), _addr(residual), _addr(weight),
                                         _addr(post_weight), _addr(gate), _addr(out),
                                         _addr(residual_out), tokens, dim, rows, float(scale),
                                         float(eps), code, _residual_code(y, residual_out), s),
              "ssd_block_norm")
    return out, residual_out


def ssd_block_norm_bwd(y, residual_out, weight, dout, dresidual_out=None, post_weight=None,
                       gate=None, scale=1.0, eps=1e-5, workspace: Workspace | None = None,
                       stream=None):
    """Gradients of ssd_block_norm from its y and residual_out, for dout and
    dresidual_out (None: zero).  Returns a dict with dy, dresidual, dweight,
    dpost_weight and dgate (None where the input is absent)."""
    code, tokens, dim, rows = _norm_args(y, weight, post_weight, gate)
    rcode = _residual_code(y, residual_out)
    dev, f32 = y.device, torch.float32
    _same(residual_out, "residual_out", y.shape, residual_out.dtype, dev, True)
    _same(dout, "dout", y.shape, y.dtype, dev, True)
    _same(dresidual_out, "dresidual_out", y.shape, residual_out.dtype, dev, True)
    lib = _lib.load()
    with _On(y, stream, (y, residual_out, weight, dout, dresidual_out, post_weight, gate)) as s:
        out = {"dy": torch.empty(y.shape, dtype=y.dtype, device=dev),
               "dresidual": torch.empty(y.shape, dtype=residual_out.dtype, device=dev),
               "dweight": torch.empty((dim,), dtype=f32, device=dev),
               "dpost_weight": None if post_weight is None else torch.empty((dim,), dtype=f32, device=dev),
               "dgate": None if gate is None else torch.empty(gate.shape, dtype=f32, device=dev)}
        ws, size, _keep = _workspace(lib.ssd_block_norm_bwd_workspace_size(tokens, dim, rows), workspace, dev)
        check(lib.ssd_block_norm_bwd(_addr(y), _addr(residual_out), _addr(weight), _addr(post_weight),
                                     _addr(gate), _addr(dout), _addr(dresidual_out), _addr(out["dy"]),
                                     _addr(out["dresidual"]), _addr(out["dweight"]),
                                     _addr(out["dpost_weight"]), _addr(out["dgate"]), tokens, dim,
                                     rows, float(scale), float(eps), code, rcode, ws, size, s),
              "ssd_block_norm_bwd")
    return out


class BlockNormFunction(torch.autograd.Function):
    """torch.autograd binding of ssd_block_norm: apply(y, residual, weight,
    post_weight, gate, scale, eps) -> (out, residual_out)."""

    @staticmethod
    def forward(ctx, y, residual, weight, post_weight=None, gate=None, scale=1.0, eps=1e-5):
        out, res = ssd_block_norm(y, residual, weight, post_weight, gate, scale, eps)
        ctx.save_for_backward(y, res, weight, post_weight, gate)
        ctx.scalars = (scale, eps)
        ctx.has_residual = residual is not None
        return out, res

    @staticmethod
    def backward(ctx, dout, dres):
        y, res, weight, post_weight, gate = ctx.saved_tensors
        g = ssd_block_norm_bwd(y, res, weight, dout.contiguous(), dres.contiguous(), post_weight,
                               gate, *ctx.scalars)
        return (g["dy"], g["dresidual"] if ctx.has_residual else None, g["dweight"],
                g["dpost_weight"], g["dgate"], None, None)
