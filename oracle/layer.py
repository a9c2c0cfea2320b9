"""Float64 references of the layer operators around the scan (test
infrastructure, as the rest of this package; numpy, token by token).

``conv`` / ``conv_bwd`` -- the short causal depthwise convolution; ``scan`` /
``scan_bwd`` -- the selective scan; ``block_norm`` / ``block_norm_bwd`` -- the
norms between blocks.  The gradients are written from the adjoint formulas
and pinned by central differences in the tests.
"""
from __future__ import annotations

import numpy as np

from . import _f64


def _sigmoid(v):
    return 0.5 * (1.0 + np.tanh(0.5 * v))


def _silu(v):
    return v * _sigmoid(v)


def _silu_grad(v):
    s = _sigmoid(v)
    return s + v * s * (1.0 - s)


def conv(x, weight, bias=None, init=None, silu=True):
    """x [B, L, D], weight [D, W], init [B, W-1, D] -> (y, last W-1 tokens)."""
    x, weight, bias, init = _f64(x), _f64(weight), _f64(bias), _f64(init)
    B, L, D = x.shape
    W = weight.shape[1]
    full = np.concatenate([np.zeros((B, W - 1, D)) if init is None else init, x], 1)
    pre = np.zeros_like(x)
    for t in range(L):
        for k in range(W):
            pre[:, t] += weight[:, k] * full[:, t + k]
    if bias is not None:
        pre += bias
    return (_silu(pre) if silu else pre), full[:, L:].copy()


def conv_bwd(x, weight, dy, bias=None, init=None, dfinal=None, silu=True):
    x, weight, bias, init = _f64(x), _f64(weight), _f64(bias), _f64(init)
    dy, dfinal = _f64(dy), _f64(dfinal)
    B, L, D = x.shape
    W = weight.shape[1]
    full = np.concatenate([np.zeros((B, W - 1, D)) if init is None else init, x], 1)
    pre, _ = conv(x, weight, bias, init, silu=False)
    dpre = dy * _silu_grad(pre) if silu else dy
    dfull = np.zeros_like(full)
    if dfinal is not None:
        dfull[:, L:] += dfinal
    dw = np.zeros_like(weight)
    for t in range(L):
        for k in range(W):
            dfull[:, t + k] += weight[:, k] * dpre[:, t]
            dw[:, k] += (dpre[:, t] * full[:, t + k]).sum(0)
    return {"dx": dfull[:, W - 1:], "dweight": dw, "dbias": dpre.sum((0, 1)), "dinit": dfull[:, :W - 1]}


def _delta(dt, dt_bias, softplus):
    raw = dt if dt_bias is None else dt + dt_bias
    return raw, (np.logaddexp(0.0, raw) if softplus else raw)


def _per_channel(m, dim):
    """[B, L, G, N] -> [B, L, dim, N], each group's row for its channels."""
    return np.repeat(m, dim // m.shape[2], axis=2)


def scan(u, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, softplus=True, init=None):
    """u, dt, z [B, L, dim]; A [dim, N]; Bm, Cm [B, L, G, N]; init [B, dim, N].
    Returns (y, states [B, L + 1, dim, N]); states[:, t] is the one before
    token t."""
    u, dt, A, Bm, Cm, D, z, dt_bias, init = map(_f64, (u, dt, A, Bm, Cm, D, z, dt_bias, init))
    B, L, dim = u.shape
    _, delta = _delta(dt, dt_bias, softplus)
    Bc, Cc = _per_channel(Bm, dim), _per_channel(Cm, dim)
    h = np.zeros((B, L + 1, dim, A.shape[1]))
    if init is not None:
        h[:, 0] = init
    y = np.zeros_like(u)
    for t in range(L):
        h[:, t + 1] = np.exp(delta[:, t, :, None] * A) * h[:, t] + (delta[:, t] * u[:, t])[..., None] * Bc[:, t]
        y[:, t] = (h[:, t + 1] * Cc[:, t]).sum(-1)
    if D is not None:
        y += D * u
    if z is not None:
        y *= _silu(z)
    return y, h


def scan_bwd(u, dt, A, Bm, Cm, dy, D=None, z=None, dt_bias=None, softplus=True, init=None, dfinal=None):
    u, dt, A, Bm, Cm, D, z, dt_bias, init, dy, dfinal = map(
        _f64, (u, dt, A, Bm, Cm, D, z, dt_bias, init, dy, dfinal))
    B, L, dim = u.shape
    G, N = Bm.shape[2], Bm.shape[3]
    raw, delta = _delta(dt, dt_bias, softplus)
    _, h = scan(u, dt, A, Bm, Cm, None, None, dt_bias, softplus, init)
    Bc, Cc = _per_channel(Bm, dim), _per_channel(Cm, dim)
    Dv = np.zeros(dim) if D is None else D
    gate = np.ones_like(u) if z is None else _silu(z)
    dyy = dy * gate
    out = {k: np.zeros_like(u) for k in ("du", "ddt", "dz")}
    out.update(dA=np.zeros_like(A), dB=np.zeros_like(Bm), dC=np.zeros_like(Cm))
    e = np.zeros((B, dim, N)) if dfinal is None else dfinal.copy()
    for t in range(L - 1, -1, -1):
        a = np.exp(delta[:, t, :, None] * A)
        e = e + dyy[:, t, :, None] * Cc[:, t]
        decayed = a * h[:, t]
        eb = (e * Bc[:, t]).sum(-1)
        out["du"][:, t] = delta[:, t] * eb + Dv * dyy[:, t]
        dd = u[:, t] * eb + (e * decayed * A).sum(-1)
        out["ddt"][:, t] = dd * _sigmoid(raw[:, t]) if softplus else dd
        out["dA"] += (e * decayed * delta[:, t, :, None]).sum(0)
        out["dB"][:, t] = (e * (delta[:, t] * u[:, t])[..., None]).reshape(B, G, dim // G, N).sum(2)
        out["dC"][:, t] = (dyy[:, t, :, None] * h[:, t + 1]).reshape(B, G, dim // G, N).sum(2)
        skip = (h[:, t + 1] * Cc[:, t]).sum(-1) + Dv * u[:, t]
        if z is not None:
            out["dz"][:, t] = dy[:, t] * skip * _silu_grad(z[:, t])
        e = a * e
    out["dD"] = (dyy * u).sum((0, 1))
    out["ddt_bias"] = out["ddt"].sum((0, 1))
    out["dinit"] = e
    return out


def _rms(v, eps):
    return v / np.sqrt((v * v).mean(-1, keepdims=True) + eps)


def _rms_bwd(g, v, eps):
    rs = 1.0 / np.sqrt((v * v).mean(-1, keepdims=True) + eps)
    return rs * g - v * rs ** 3 * (g * v).mean(-1, keepdims=True)


def _gate_rows(gate, tokens):
    return np.repeat(gate, tokens // gate.shape[0], axis=0)


def block_norm(y, residual, weight, post_weight=None, gate=None, scale=1.0, eps=1e-5):
    """y, residual [T, D]; gate [rows, D] -> (out, residual after the block)."""
    y, residual, weight, post_weight, gate = map(_f64, (y, residual, weight, post_weight, gate))
    p = y if post_weight is None else _rms(y, eps) * post_weight
    if gate is not None:
        p = p * _gate_rows(gate, y.shape[0])
    r = scale * p if residual is None else residual + scale * p
    return _rms(r, eps) * weight, r


def block_norm_bwd(y, r, weight, dout, dr=None, post_weight=None, gate=None, scale=1.0, eps=1e-5):
    """r: the residual after the block."""
    y, r, weight, dout, dr, post_weight, gate = map(_f64, (y, r, weight, dout, dr, post_weight, gate))
    gr = _rms_bwd(dout * weight, r, eps)
    if dr is not None:
        gr = gr + dr
    p = y if post_weight is None else _rms(y, eps) * post_weight
    dp = scale * gr if gate is None else scale * gr * _gate_rows(gate, y.shape[0])
    out = {"dresidual": gr, "dweight": (dout * _rms(r, eps)).sum(0), "dy": dp}
    if gate is not None:
        out["dgate"] = scale * (gr * p).reshape(gate.shape[0], -1, y.shape[1]).sum(1)
    if post_weight is not None:
        out["dpost_weight"] = (dp * _rms(y, eps)).sum(0)
        out["dy"] = _rms_bwd(dp * post_weight, y, eps)
    return out
