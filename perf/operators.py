"""Cases for the operators around the scan: the short causal convolution, the
selective scan and the block norm, in their forms for training, prompts and
single tokens.

``run`` computes a case in plain torch operations (32-bit arithmetic, one
rounding at the end) or, with ``own`` set, through the framework's calls.
Every case is one call a layer makes: ``listed`` holds the sizes of a 2.7B
layer (2560 model channels, 5120 inner channels, 128 states of one group
beside them in the convolution), a long prompt and small or ragged ones.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def conv_case(op, batch, seqlen, dim, width, dtype, *, act=True, bias=True, carry=False, row=0, **name):
    """row: elements between tokens of x (0: dim, contiguous)."""
    return dict(name, op=op, batch=batch, seqlen=seqlen, dim=dim, width=width, dtype=dtype, act=act,
                bias=bias, carry=carry, row=row or dim)


def scan_case(op, batch, seqlen, dim, dstate, ngroups, dtype, *, gated=True, carry=False, row=0, **name):
    """row: elements between tokens of u and z (0: dim, contiguous)."""
    return dict(name, op=op, batch=batch, seqlen=seqlen, dim=dim, dstate=dstate, ngroups=ngroups,
                dtype=dtype, gated=gated, carry=carry, row=row or dim)


def norm_case(op, tokens, dim, dtype, residual, *, gate_rows=0, post=True, **name):
    """gate_rows: rows of the gate (0: none), each for tokens / gate_rows tokens."""
    return dict(name, op=op, tokens=tokens, dim=dim, dtype=dtype, residual=residual,
                gate_rows=gate_rows, post=post)


def listed():
    return [
        # a prompt batch's x, B and C slice of the input projection, 5120 + 2 x 128 channels
        conv_case("conv", 4, 4096, 5376, 4, "bf16", row=10576, name="conv_prompt"),
        # the same slice in training, backward
        conv_case("conv_grad", 4, 4096, 5376, 4, "bf16", row=10576, name="conv_train"),
        # a chunk of a prompt in 32 bits, odd sizes, continued from the chunk before
        conv_case("conv", 3, 1531, 1537, 3, "f32", bias=False, carry=True, name="conv_ragged_f32"),
        # 128 sequences, one token each
        conv_case("conv_token", 128, 1, 5376, 4, "bf16", row=10576, name="conv_token"),
        # a prompt batch through one selective layer, u and z slices of one projection
        scan_case("scan", 4, 4096, 5120, 16, 1, "bf16", row=10240, name="scan_prompt"),
        # one long prompt, continued from a state
        scan_case("scan", 1, 32768, 4096, 16, 1, "bf16", carry=True, name="scan_long"),
        # few channels in two groups, odd length, 32 bits
        scan_case("scan", 2, 1531, 500, 8, 2, "f32", gated=False, carry=True, name="scan_ragged_f32"),
        # a training step of one layer: the forward that keeps what its backward needs, and the backward
        scan_case("scan_grad", 2, 4096, 5120, 16, 1, "bf16", row=10240, name="scan_train"),
        # 128 sequences, one token each
        scan_case("scan_token", 128, 1, 5120, 16, 1, "bf16", row=10240, name="scan_token"),
        # between two blocks of a prompt or training batch: 32-bit residual, one gate row per sequence
        norm_case("norm", 16384, 2560, "bf16", "f32", gate_rows=4, name="norm_prompt"),
        norm_case("norm_grad", 16384, 2560, "bf16", "f32", gate_rows=4, name="norm_train"),
        # between two blocks, eight sequences with one token each
        norm_case("norm", 8, 2560, "bf16", "bf16", name="norm_token"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "conv_grad", "conv_token", "scan", "scan", "scan_grad", "scan_token",
                     "norm", "norm_grad"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("conv"):
        dim = _log(rng, 64, 8192)
        if rng.random() < 0.6:
            dim = -(-dim // 64) * 64
        batch, seqlen = _log(rng, 1, 8), _log(rng, 1, 32768)
        if op == "conv_token":
            batch, seqlen = _log(rng, 1, 512), 1
        else:
            seqlen = max(1, min(seqlen, 4 * 4096 * 5376 // 2 // (batch * dim)))
        row = dim if rng.random() < 0.5 else dim + 8 * rng.randint(1, 700)
        return conv_case(op, batch, seqlen, dim, rng.randint(2, 4), dtype, act=rng.random() < 0.8,
                         bias=rng.random() < 0.7, carry=rng.random() < 0.5, row=row)
    if op.startswith("scan"):
        ngroups = rng.choice([1, 1, 1, 2, 4])
        dim = ngroups * _log(rng, 16, 5120 // ngroups)
        if rng.random() < 0.6:
            dim = -(-dim // (64 * ngroups)) * 64 * ngroups
        dstate = rng.choice([16, 16, 16, 8, 32, 64, 5])
        batch, seqlen = _log(rng, 1, 8), _log(rng, 1, 32768)
        if op == "scan_token":
            batch, seqlen = _log(rng, 1, 512), 1
        else:
            most = 2 * 4096 * 5120 * 16 // (2 if dtype == "f32" else 1)
            seqlen = max(1, min(seqlen, most // (batch * dim * dstate)))
        row = dim if rng.random() < 0.5 else dim + 8 * rng.randint(1, 700)
        return scan_case(op, batch, seqlen, dim, dstate, ngroups, dtype, gated=rng.random() < 0.7,
                         carry=rng.random() < 0.5, row=row)
    dim = _log(rng, 64, 8192)
    if rng.random() < 0.7:
        dim = -(-dim // 64) * 64
    gate = rng.choice(["none", "channel", "sequence", "token"])
    sequences = _log(rng, 1, 8)
    tokens = sequences * max(1, min(_log(rng, 1, 32768), 16384 * 2560 // 2 // (sequences * dim)))
    rows = {"none": 0, "channel": 1, "sequence": sequences, "token": tokens}[gate]
    return norm_case(op, tokens, dim, dtype, rng.choice([dtype, "f32"]), gate_rows=rows,
                     post=rng.random() < 0.6)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

class _Draws:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(self, shape, dtype=torch.float32, std=1.0, mean=0.0):
        t = torch.randn(shape, generator=self.g, device="cuda", dtype=torch.float32)
        return (t * std + mean).to(dtype)

    def uniform(self, shape, lo, hi):
        return torch.rand(shape, generator=self.g, device="cuda") * (hi - lo) + lo

    def rows(self, shape, row, dtype):
        """[..., dim] values inside a wider projection output: `row` elements between rows."""
        t = torch.zeros(tuple(shape[:-1]) + (row,), device="cuda", dtype=dtype)
        v = t[..., row - shape[-1]:]
        v.copy_(self.normal(shape, dtype))
        return v


def prepare(case, seed):
    c, r = case, _Draws(seed)
    dt = DTYPES[c["dtype"]]
    s = {"case": c}
    if c["op"].startswith("conv"):
        b, L, D, W = c["batch"], c["seqlen"], c["dim"], c["width"]
        token = c["op"] == "conv_token"
        s["x"] = r.rows((b, D) if token else (b, L, D), c["row"], dt)
        s["weight"] = r.uniform((D, W), -1.0, 1.0) / math.sqrt(W)
        s["bias"] = r.uniform((D,), -0.5, 0.5) if c["bias"] else None
        s["init"] = r.normal((b, W - 1, D), dt) if c["carry"] or token else None
        if token:
            s["state_out"] = torch.empty_like(s["init"])
        if c["op"] == "conv_grad":
            s["dy"] = r.normal((b, L, D), dt)
            s["dfinal"] = r.normal((b, W - 1, D), dt) if c["carry"] else None
    elif c["op"].startswith("scan"):
        b, L, D, N, G = c["batch"], c["seqlen"], c["dim"], c["dstate"], c["ngroups"]
        token = c["op"] == "scan_token"
        lead = (b,) if token else (b, L)
        s["u"] = r.rows(lead + (D,), c["row"], dt)
        s["dt"] = r.normal(lead + (D,), dt, std=0.5)
        # softplus(dt_bias) in [1e-3, 1e-1], A in [-16, -1]
        s["dt_bias"] = torch.log(torch.expm1(torch.exp(r.uniform((D,), math.log(1e-3), math.log(1e-1)))))
        s["A"] = -torch.exp(r.uniform((D, N), 0.0, math.log(16.0)))
        s["B"] = r.normal(lead + (G, N), dt, std=1.0 / math.sqrt(N))
        s["C"] = r.normal(lead + (G, N), dt, std=1.0 / math.sqrt(N))
        s["D"] = r.normal((D,), std=0.1, mean=1.0)
        s["z"] = r.rows(lead + (D,), c["row"], dt) if c["gated"] else None
        s["init"] = r.normal((b, D, N), std=0.1) if c["carry"] or token else None
        if token:
            s["state_out"] = torch.empty_like(s["init"])
        if c["op"] == "scan_grad":
            s["dy"] = r.normal((b, L, D), dt)
            s["dfinal"] = r.normal((b, D, N)) if c["carry"] else None
    else:
        t, D = c["tokens"], c["dim"]
        rt = DTYPES[c["residual"]]
        s["y"] = r.normal((t, D), dt)
        s["weight"] = r.normal((D,), std=0.1, mean=1.0)
        s["post_weight"] = r.normal((D,), std=0.1, mean=1.0) if c["post"] else None
        s["gate"] = r.normal((c["gate_rows"], D), std=0.3, mean=0.7) if c["gate_rows"] else None
        s["scale"] = 0.25
        s["eps"] = 1e-5
        s["residual"] = r.normal((t, D), rt, std=2.0)  # before the block, or (backward) after it
        if c["op"] == "norm_grad":
            s["dout"] = r.normal((t, D), dt)
            s["dresidual"] = r.normal((t, D), rt)
    return s


# --------------------------------------------------------------------------
# the plain forms
# --------------------------------------------------------------------------

def _f(t):
    return None if t is None else t.float()


def _silu(v):
    return v / (1.0 + torch.exp(-v))


def _dsilu(v):
    s = 1.0 / (1.0 + torch.exp(-v))
    return s * (1.0 + v * (1.0 - s))


def _padded(x, init, width):
    """x with the width - 1 tokens before it (zeros without a carried state)."""
    if init is None:
        init = x.new_zeros((x.shape[0], width - 1, x.shape[2]))
    return torch.cat([init, x], 1)


def _windows(x, width):
    """[batch, seqlen, dim, width]: each token's window, oldest first."""
    return x.unfold(1, width, 1)


def plain_conv(s):
    c = s["case"]
    xp = _padded(_f(s["x"]), _f(s["init"]), c["width"])
    pre = (_windows(xp, c["width"]) * s["weight"]).sum(-1)
    if s["bias"] is not None:
        pre = pre + s["bias"]
    y = _silu(pre) if c["act"] else pre
    dt = s["x"].dtype
    return y.to(dt), xp[:, xp.shape[1] - (c["width"] - 1):].to(dt)


def plain_conv_token(s):
    c = s["case"]
    xp = torch.cat([_f(s["init"]), _f(s["x"]).unsqueeze(1)], 1)
    pre = (xp.transpose(1, 2) * s["weight"]).sum(-1)
    if s["bias"] is not None:
        pre = pre + s["bias"]
    y = _silu(pre) if c["act"] else pre
    return y.to(s["x"].dtype), xp[:, 1:].to(s["x"].dtype)


def plain_conv_grad(s):
    c = s["case"]
    W = c["width"]
    win = _windows(_padded(_f(s["x"]), _f(s["init"]), W), W)
    dpre = _f(s["dy"])
    if c["act"]:
        pre = (win * s["weight"]).sum(-1)
        if s["bias"] is not None:
            pre = pre + s["bias"]
        dpre = dpre * _dsilu(pre)
    dw = (win * dpre.unsqueeze(-1)).sum((0, 1))
    db = dpre.sum((0, 1)) if s["bias"] is not None else None
    ahead = torch.nn.functional.pad(dpre, (0, 0, W - 1, W - 1))
    dxp = (_windows(ahead, W) * s["weight"].flip(-1)).sum(-1)  # of (init | x)
    if s["dfinal"] is not None:
        dxp[:, dxp.shape[1] - (W - 1):] += _f(s["dfinal"])
    dt = s["x"].dtype
    return {"dx": dxp[:, W - 1:].to(dt), "dweight": dw, "dbias": db,
            "dinit": dxp[:, :W - 1].to(dt) if s["init"] is not None else None}


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1 from h = 0, by doubling."""
    step = 1
    while step < a.shape[1]:
        b = torch.cat([b[:, :step], b[:, step:] + a[:, step:] * b[:, :-step]], 1)
        a = torch.cat([a[:, :step], a[:, step:] * a[:, :-step]], 1)
        step *= 2
    return b


def _softplus(v):
    return torch.clamp(v, min=0.0) + torch.log1p(torch.exp(-torch.abs(v)))


def _scan_parts(s):
    """delta [b,L,D], decays a and inputs b as [b,L,G,K,N], states h alike."""
    c = s["case"]
    G, N = c["ngroups"], c["dstate"]
    u, raw = _f(s["u"]), _f(s["dt"]) + s["dt_bias"]
    delta = _softplus(raw)
    lead = u.shape[:2]
    A = s["A"].view(G, -1, N)
    B, C = _f(s["B"]).unsqueeze(3), _f(s["C"]).unsqueeze(3)
    per = lead + (G, -1, 1)
    a = torch.exp(delta.view(per) * A)
    b = (delta * u).view(per) * B
    if s["init"] is not None:
        b[:, 0] += a[:, 0] * s["init"].view(-1, G, A.shape[1], N)
    return u, raw, delta, A, B, C, a, _scan(a, b)


def plain_scan(s):
    u, _, _, _, _, C, _, h = _scan_parts(s)
    y = (h * C).sum(-1).view(u.shape) + s["D"] * u
    if s["z"] is not None:
        y = y * _silu(_f(s["z"]))
    return y.to(s["u"].dtype), h[:, -1].reshape(h.shape[0], -1, h.shape[-1])


def plain_scan_token(s):
    c = s["case"]
    G, N = c["ngroups"], c["dstate"]
    u = _f(s["u"])
    delta = _softplus(_f(s["dt"]) + s["dt_bias"])
    per = (u.shape[0], G, -1, 1)
    h = torch.exp(delta.view(per) * s["A"].view(G, -1, N)) * s["init"].view(u.shape[0], G, -1, N)
    h = h + (delta * u).view(per) * _f(s["B"]).unsqueeze(2)
    y = (h * _f(s["C"]).unsqueeze(2)).sum(-1).view(u.shape) + s["D"] * u
    if s["z"] is not None:
        y = y * _silu(_f(s["z"]))
    return y.to(s["u"].dtype), h.reshape(s["init"].shape)


def plain_scan_grad(s):
    u, raw, delta, A, B, C, a, h = _scan_parts(s)
    per = u.shape[:2] + (A.shape[0], -1, 1)
    skip = (h * C).sum(-1).view(u.shape) + s["D"] * u
    dy = _f(s["dy"])
    y, dz = skip, None
    if s["z"] is not None:
        z = _f(s["z"])
        y, dz, dy = skip * _silu(z), dy * skip * _dsilu(z), dy * _silu(z)
    # the states' gradients: e_t = C_t dy_t + a_{t+1} e_{t+1}, from the last token back
    e = dy.view(per) * C
    if s["dfinal"] is not None:
        e[:, -1] += s["dfinal"].view(e[:, -1].shape)
    ahead = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    e = _scan(ahead.flip(1), e.flip(1)).flip(1)
    first = torch.zeros_like(h[:, :1]) if s["init"] is None else s["init"].view(h[:, :1].shape)
    decayed = a * torch.cat([first, h[:, :-1]], 1)  # a_t h_{t-1}
    eb = (e * B).sum(-1).view(u.shape)
    q = e * decayed
    ddelta = u * eb + (q * A).sum(-1).view(u.shape)
    ddt = ddelta / (1.0 + torch.exp(-raw))
    dt = s["u"].dtype
    lead = u.shape[0], u.shape[2]
    return {"y": y.to(dt), "final_state": h[:, -1].reshape(lead + (-1,)),
            "du": (delta * eb + s["D"] * dy).to(dt), "ddt": ddt.to(dt),
            "dA": (q * delta.view(per)).sum((0, 1)).reshape(s["A"].shape),
            "dB": (e * (delta * u).view(per)).sum(3).to(dt), "dC": (h * dy.view(per)).sum(3).to(dt),
            "dD": (dy * u).sum((0, 1)), "dz": None if dz is None else dz.to(dt),
            "ddt_bias": ddt.sum((0, 1)),
            "dinit": None if s["init"] is None else (a * e)[:, 0].reshape(lead + (-1,))}


def _rms(v, eps):
    return v / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)


def _rms_back(g, xhat, v, eps):
    """Gradient of v from g, that of xhat = _rms(v)."""
    return (g - xhat * (g * xhat).mean(-1, keepdim=True)) / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)


def _gate(s):
    """One gate row for each token, or 1."""
    if s["gate"] is None:
        return 1.0
    return s["gate"].repeat_interleave(s["y"].shape[0] // s["gate"].shape[0], 0)


def plain_norm(s):
    p = _f(s["y"])
    if s["post_weight"] is not None:
        p = _rms(p, s["eps"]) * s["post_weight"]
    r = _f(s["residual"]) + s["scale"] * (_gate(s) * p)
    return (_rms(r, s["eps"]) * s["weight"]).to(s["y"].dtype), r.to(s["residual"].dtype)


def plain_norm_grad(s):
    y, r, dout = _f(s["y"]), _f(s["residual"]), _f(s["dout"])
    rhat = _rms(r, s["eps"])
    gr = _f(s["dresidual"]) + _rms_back(dout * s["weight"], rhat, r, s["eps"])
    p = y
    if s["post_weight"] is not None:
        yhat = _rms(y, s["eps"])
        p = yhat * s["post_weight"]
    dp = s["scale"] * (_gate(s) * gr)
    dgate = None
    if s["gate"] is not None:
        dgate = s["scale"] * (gr * p).view(s["gate"].shape[0], -1, y.shape[1]).sum(1)
    dy, dpost = dp, None
    if s["post_weight"] is not None:
        dpost = (dp * yhat).sum(0)
        dy = _rms_back(dp * s["post_weight"], yhat, y, s["eps"])
    return {"dy": dy.to(s["y"].dtype), "dresidual": gr.to(s["residual"].dtype),
            "dweight": (dout * rhat).sum(0), "dpost_weight": dpost, "dgate": dgate}


PLAIN = {"conv": plain_conv, "conv_grad": plain_conv_grad, "conv_token": plain_conv_token,
         "scan": plain_scan, "scan_grad": plain_scan_grad, "scan_token": plain_scan_token,
         "norm": plain_norm, "norm_grad": plain_norm_grad}


# --------------------------------------------------------------------------
# the framework's calls
# --------------------------------------------------------------------------

def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return PLAIN[op](s)
    import state_space_sequence_cumsum_gb300 as ssd
    act = "silu" if s["case"].get("act") else None
    if op == "conv":
        return ssd.ssd_causal_conv(s["x"], s["weight"], s["bias"], activation=act,
                                   initial_state=s["init"], return_final_state=True)
    if op == "conv_token":
        return ssd.ssd_causal_conv_step(s["x"], s["weight"], s["init"], s["bias"], activation=act,
                                        state_out=s["state_out"])
    if op == "conv_grad":
        return ssd.ssd_causal_conv_bwd(s["x"], s["weight"], s["dy"], s["bias"], activation=act,
                                       initial_state=s["init"], dfinal=s["dfinal"],
                                       want_dinit=s["init"] is not None)
    if op == "scan":
        return ssd.ssd_selective_scan(s["u"], s["dt"], s["A"], s["B"], s["C"], s["D"], z=s["z"],
                                      dt_bias=s["dt_bias"], initial_state=s["init"])[:2]
    if op == "scan_token":
        return ssd.ssd_selective_scan_step(s["u"], s["dt"], s["A"], s["B"], s["C"], s["D"],
                                           s["init"], z=s["z"], dt_bias=s["dt_bias"],
                                           state_out=s["state_out"])
    if op == "scan_grad":
        y, final, kept = ssd.ssd_selective_scan(s["u"], s["dt"], s["A"], s["B"], s["C"], s["D"],
                                                z=s["z"], dt_bias=s["dt_bias"],
                                                initial_state=s["init"], return_chunk_states=True)
        grads = ssd.ssd_selective_scan_bwd(s["u"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["dy"],
                                           z=s["z"], dt_bias=s["dt_bias"], initial_state=s["init"],
                                           dfinal=s["dfinal"], chunk_states=kept,
                                           want_dinit=s["init"] is not None)
        return {"y": y, "final_state": final, **grads}
    if op == "norm":
        return ssd.ssd_block_norm(s["y"], s["residual"], s["weight"], post_weight=s["post_weight"],
                                  gate=s["gate"], scale=s["scale"], eps=s["eps"])
    return ssd.ssd_block_norm_bwd(s["y"], s["residual"], s["weight"], s["dout"], s["dresidual"],
                                  post_weight=s["post_weight"], gate=s["gate"], scale=s["scale"],
                                  eps=s["eps"])


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"].startswith("conv"):
        b, L, D, W = c["batch"], c["seqlen"], c["dim"], c["width"]
        tokens, state = b * L * D, b * (W - 1) * D * e
        params = 4 * D * (W + int(c["bias"]))
        carried = state * int(c["carry"] or c["op"] == "conv_token")
        act = 5 if c["act"] else 0
        if c["op"] == "conv_grad":
            return {"bytes": 3 * tokens * e + 2 * params + 3 * carried,
                    "flops": tokens * (6 * W + 2 * act)}
        return {"bytes": 2 * tokens * e + params + carried + state, "flops": tokens * (2 * W + act)}
    if c["op"].startswith("scan"):
        b, L, D, N, G = c["batch"], c["seqlen"], c["dim"], c["dstate"], c["ngroups"]
        tokens, bc, state = b * L * D * e, 2 * b * L * G * N * e, 4 * b * D * N
        gated = int(c["gated"])
        params = 4 * D * (N + 2)
        carried = state * int(c["carry"] or c["op"] == "scan_token")
        entries = b * L * D * N
        forward = {"bytes": (3 + gated) * tokens + bc + params + carried + state,
                   "flops": 7 * entries + 20 * b * L * D}
        if c["op"] != "scan_grad":
            return forward
        # the forward, then the backward: u, dt, z, dy, B, C in; their gradients out
        return {"bytes": forward["bytes"] + (5 + 2 * gated) * tokens + 2 * bc + 2 * params + 3 * carried,
                "flops": forward["flops"] + 25 * entries + 40 * b * L * D}
    t, D = c["tokens"], c["dim"]
    er = 2 if c["residual"] == "bf16" else 4
    params = 4 * D * (1 + int(c["post"]) + c["gate_rows"])
    if c["op"] == "norm":
        return {"bytes": t * D * (2 * e + 2 * er) + params, "flops": t * D * 12}
    return {"bytes": t * D * (3 * e + 3 * er) + 2 * params, "flops": t * D * 25}


# --------------------------------------------------------------------------
# 64 bits, from the definitions
# --------------------------------------------------------------------------

def _exact_conv(x, weight, bias, init, act):
    """Each output token from its own window; (y, final)."""
    W = weight.shape[1]
    if init is None:
        init = x.new_zeros((x.shape[0], W - 1, x.shape[2]))
    full = torch.cat([init, x], 1)
    L = x.shape[1]
    y = torch.zeros_like(x)
    for k in range(W):
        y = y + full[:, k:k + L] * weight[:, k]
    if bias is not None:
        y = y + bias
    if act:
        y = y * torch.sigmoid(y)
    return y, full[:, L:]


def _exact_scan(u, dt, A, B, C, D, z, dt_bias, init):
    """The recurrence token by token; (y, final)."""
    b, L, dim = u.shape
    G, N = B.shape[2], B.shape[3]
    delta = torch.nn.functional.softplus(dt + dt_bias, threshold=100.0)
    A4 = A.view(1, G, dim // G, N)
    h = u.new_zeros((b, G, dim // G, N)) if init is None else init.view(b, G, dim // G, N)
    ys = []
    for d_t, u_t, B_t, C_t in zip(delta.unbind(1), u.unbind(1), B.unbind(1), C.unbind(1)):
        d4 = d_t.reshape(b, G, dim // G, 1)
        h = torch.exp(d4 * A4) * h + d4 * u_t.reshape(b, G, dim // G, 1) * B_t.unsqueeze(2)
        ys.append(torch.einsum("bgkn,bgn->bgk", h, C_t).reshape(b, dim))
    y = torch.stack(ys, 1) + D * u
    if z is not None:
        y = y * (z * torch.sigmoid(z))
    return y, h.reshape(b, dim, N)


def _exact_norm(y, residual, weight, post_weight, gate, scale, eps):
    p = y
    if post_weight is not None:
        p = p * torch.rsqrt(torch.mean(torch.square(p), 1, keepdim=True) + eps) * post_weight
    if gate is not None:
        p = (p.view(gate.shape[0], -1, p.shape[1]) * gate.unsqueeze(1)).reshape(p.shape)
    r = residual + scale * p
    return r * torch.rsqrt(torch.mean(torch.square(r), 1, keepdim=True) + eps) * weight, r


def exact(case, seed):
    """The definitions in 64 bits; gradients by differentiating them."""
    c, op = case, case["op"]
    s = prepare(case, seed)
    # the gradient keeps about six 64-bit values of every state
    if op == "scan_grad" and c["batch"] * c["seqlen"] * c["dim"] * c["dstate"] > 800_000_000:
        return None
    d = {k: v.double() if isinstance(v, torch.Tensor) and k != "state_out" else v for k, v in s.items()}
    if op == "conv":
        return _exact_conv(d["x"], d["weight"], d["bias"], d["init"], c["act"])
    if op == "conv_token":
        y, final = _exact_conv(d["x"].unsqueeze(1), d["weight"], d["bias"], d["init"], c["act"])
        return y[:, 0], final
    if op == "scan":
        return _exact_scan(d["u"], d["dt"], d["A"], d["B"], d["C"], d["D"], d["z"], d["dt_bias"], d["init"])
    if op == "scan_token":
        one = {k: d[k].unsqueeze(1) if d[k] is not None else None for k in ("u", "dt", "B", "C", "z")}
        y, final = _exact_scan(one["u"], one["dt"], d["A"], one["B"], one["C"], d["D"], one["z"],
                               d["dt_bias"], d["init"])
        return y[:, 0], final
    if op == "norm":
        return _exact_norm(d["y"], d["residual"], d["weight"], d["post_weight"], d["gate"], d["scale"], d["eps"])

    def gradients(names, outputs, cotangents):
        have = [n for n in names if d[n] is not None]
        pairs = [(o, g) for o, g in zip(outputs, cotangents) if g is not None]
        got = torch.autograd.grad([o for o, _ in pairs], [d[n] for n in have], [g for _, g in pairs])
        return {**dict.fromkeys(names), **dict(zip(have, got))}

    names = {"conv_grad": ["x", "weight", "bias", "init"],
             "scan_grad": ["u", "dt", "A", "B", "C", "D", "z", "dt_bias", "init"],
             "norm_grad": ["y", "weight", "post_weight", "gate"]}[op]
    for n in names:
        if d[n] is not None:
            d[n].requires_grad_(True)
    if op == "conv_grad":
        out = _exact_conv(d["x"], d["weight"], d["bias"], d["init"], c["act"])
        g = gradients(names, out, (d["dy"], d["dfinal"]))
        return {"dx": g["x"], "dweight": g["weight"], "dbias": g["bias"], "dinit": g["init"]}
    if op == "scan_grad":
        out = _exact_scan(d["u"], d["dt"], d["A"], d["B"], d["C"], d["D"], d["z"], d["dt_bias"], d["init"])
        g = gradients(names, out, (d["dy"], d["dfinal"]))
        return {"y": out[0].detach(), "final_state": out[1].detach(), "du": g["u"], "ddt": g["dt"],
                "dA": g["A"], "dB": g["B"], "dC": g["C"], "dD": g["D"], "dz": g["z"],
                "ddt_bias": g["dt_bias"], "dinit": g["init"]}
    # the backward is given the residual after the block: the block's output is what went into it
    first = d["residual"].detach()
    p, r = _exact_norm(d["y"], torch.zeros_like(first), d["weight"].detach(), d["post_weight"], d["gate"],
                       d["scale"], d["eps"])
    before = (first - r).detach().requires_grad_(True)
    d["before"] = before
    out = _exact_norm(d["y"], before, d["weight"], d["post_weight"], d["gate"], d["scale"], d["eps"])
    g = gradients(names + ["before"], out, (d["dout"], d["dresidual"]))
    return {"dy": g["y"], "dresidual": g["before"], "dweight": g["weight"],
            "dpost_weight": g["post_weight"], "dgate": g["gate"]}
