"""Cases for the 8-bit projections around the scan and for the optimiser's step:
values quantised in blocks of 128, products of such matrices, a layer's
projection with its gradients, and AdamW over many tensors with its states in
32 bits or in 8.

``run`` computes a case in plain torch operations (32-bit arithmetic, one
rounding at the end) or, with ``own`` set, through the framework's calls.
``listed`` holds the sizes of a 2.7B layer (2560 model channels, 10576 outputs
of its input projection, 5120 inner channels), small and ragged ones.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn
BLOCK = 128       # values of a row that share a scale; rows too, in a tile
STATES = 256      # values of an optimiser's 8-bit state that share a scale
TOP = 448.0       # the largest e4m3 value
LEAST = 2.0 ** -100


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def quant_case(rows, cols, dtype, *, tile=False, both=True, row=0, **name):
    """row: elements between rows of x (0: cols, contiguous); both: the transpose too."""
    return dict(name, op="quant", rows=rows, cols=cols, dtype=dtype, tile=tile, both=both, row=row or cols)


def matmul_case(m, n, k, out, *, tile=True, **name):
    """tile: b has one scale for each 128 x 128, else one for each 128 of a row."""
    return dict(name, op="matmul", m=m, n=n, k=k, out=out, tile=tile)


def proj_case(op, tokens, inputs, outputs, dtype, *, row=0, **name):
    """row: elements between tokens of x (0: inputs, contiguous)."""
    return dict(name, op=op, tokens=tokens, inputs=inputs, outputs=outputs, dtype=dtype, row=row or inputs)


def adamw_case(layers, dim, bits, grads, *, vocab=0, step=100, clip=False, **name):
    """The tensors of `layers` layers of `dim` model channels and of an embedding of `vocab` rows."""
    return dict(name, op="adamw", layers=layers, dim=dim, bits=bits, grads=grads, vocab=vocab, step=step, clip=clip)


def listed():
    return [
        # a training batch's inputs of the input projection, for the product and for the weights' gradient
        quant_case(16384, 2560, "bf16", name="quant_tokens"),
        # the input projection's weights after a step of the optimiser
        quant_case(10576, 2560, "f32", tile=True, name="quant_weights"),
        # a prompt batch times the input projection, scales as a checkpoint has them
        matmul_case(16384, 10576, 2560, "bf16", name="matmul_prompt"),
        # few channels, odd sizes, a scale for each row's blocks on both sides, 32 bits out
        matmul_case(1531, 507, 2561, "f32", tile=False, name="matmul_ragged_f32"),
        # a prompt batch through the output projection, the gated scan's output a slice of a wider buffer
        proj_case("proj", 16384, 5120, 2560, "bf16", row=10240, name="proj_prompt"),
        # eight sequences, one token each, through the input projection
        proj_case("proj", 8, 2560, 10576, "bf16", name="proj_token"),
        # 128 sequences, one token each, through the output projection
        proj_case("proj", 128, 5120, 2560, "bf16", name="proj_tokens"),
        # a training step of the input projection: weights quantised, forward, both gradients
        proj_case("proj_train", 16384, 2560, 10576, "bf16", name="proj_train"),
        # the same of a small layer, odd sizes, 32 bits
        proj_case("proj_train", 701, 517, 1001, "f32", name="proj_train_ragged_f32"),
        # the optimiser's step over six layers, states in 32 bits
        adamw_case(6, 2560, 32, "f32", name="adamw_f32"),
        # the same tensors with bf16 gradients and 8-bit states
        adamw_case(6, 2560, 8, "bf16", clip=True, name="adamw_8bit"),
        # a model of two narrow layers
        adamw_case(2, 128, 32, "f32", vocab=64, name="adamw_small"),
    ]


MOST_FLOPS = 2 * 16384 * 10576 * 2560
MOST_PARAMETERS = 240_000_000


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo=64, hi=10576):
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.4 else -(-n // 64) * 64


def draw(rng):
    op = rng.choice(["quant", "matmul", "proj", "proj", "proj_train", "adamw"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "adamw":
        dim, bits = _log(rng, 16, 2560), rng.choice([8, 32])
        most = max(1, MOST_PARAMETERS // (7 * dim * dim + 2000 * dim))
        return adamw_case(min(most, _log(rng, 1, 48)), dim, bits, dtype, step=_log(rng, 1, 100000),
                          vocab=rng.choice([0, 0, 64, 1003]), clip=rng.random() < 0.5)
    if op == "quant":
        cols = _width(rng)
        rows = min(_log(rng, 1, 16384), 16384 * 2560 // cols)
        tile = rng.random() < 0.4
        row = cols if tile or rng.random() < 0.5 else cols + 8 * rng.randint(1, 700)
        return quant_case(rows, cols, dtype, tile=tile, both=rng.random() < 0.7, row=row)
    n, k = _width(rng), _width(rng)
    m = min(_log(rng, 1, 16384), MOST_FLOPS // (2 * n * k))
    if op == "matmul":
        return matmul_case(m, n, k, dtype, tile=rng.random() < 0.7)
    row = k if rng.random() < 0.5 else k + 8 * rng.randint(1, 700)
    return proj_case(op, m, k, n, dtype, row=row)


def shapes(case):
    """The tensors of an optimiser's step: those of a layer with 2 * dim inner
    channels in heads of 64 and 128 states."""
    dim, inner, dstate = case["dim"], 2 * case["dim"], 128
    heads = -(-inner // 64)
    mixed = inner + 2 * dstate
    layer = [(inner + mixed + heads, dim), (mixed, 4), (mixed,), (heads,), (heads,), (heads,), (inner,), (dim, inner),
             (dim,)]
    return layer * case["layers"] + ([(case["vocab"], dim), (dim,)] if case["vocab"] else [])


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

    def tokens(self, rows, cols, dtype):
        """Activations: channels of very different sizes, some tokens larger than the rest."""
        sizes = torch.exp(self.normal((cols,), std=1.0)) * torch.exp(self.normal((rows, 1), std=0.5))
        return (self.normal((rows, cols)) * sizes).to(dtype)

    def rows(self, values, row):
        """The values inside a wider buffer: `row` elements between rows."""
        t = torch.zeros((values.shape[0], row), device="cuda", dtype=values.dtype)
        v = t[:, row - values.shape[1]:]
        v.copy_(values)
        return v


def _up(n, to):
    return -(-n // to) * to


def _bytes16(q):
    """8-bit values with rows that start on 16 bytes."""
    t = torch.zeros((q.shape[0], _up(q.shape[1], 16)), device="cuda", dtype=q.dtype)
    t[:, :q.shape[1]] = q
    return t[:, :q.shape[1]]


def _checkpoint(w, tile):
    """8-bit weights and scales (the largest value of a block over 448) as a program has them in hand."""
    b = _blocks(w, tile).abs().amax((1, 3))
    scale = torch.clamp(b, min=1e-12) / TOP
    return _bytes16((w / _spread(scale, w, tile)).to(E4M3)), scale


def prepare(case, seed):
    c, r = case, _Draws(seed)
    s = {"case": c}
    if c["op"] == "quant":
        x = r.tokens(c["rows"], c["cols"], torch.float32)
        s["x"] = r.rows((x / math.sqrt(c["cols"]) if c["tile"] else x).to(DTYPES[c["dtype"]]), c["row"])
    elif c["op"] == "matmul":
        s["a"], s["a_scale"] = _checkpoint(r.tokens(c["m"], c["k"], torch.float32), False)
        s["b"], s["b_scale"] = _checkpoint(r.normal((c["n"], c["k"]), std=1.0 / math.sqrt(c["k"])), c["tile"])
    elif c["op"] in ("proj", "proj_train"):
        dt = DTYPES[c["dtype"]]
        s["x"] = r.rows(r.tokens(c["tokens"], c["inputs"], dt), c["row"])
        w = r.normal((c["outputs"], c["inputs"]), std=1.0 / math.sqrt(c["inputs"]))
        if c["op"] == "proj":
            s["w"], s["w_scale"] = _checkpoint(w, True)
        else:
            s["weight"] = w
            s["dy"] = r.tokens(c["tokens"], c["outputs"], dt) * 1e-3
    else:
        _prepare_adamw(c, r, s)
    return s


def _prepare_adamw(c, r, s):
    """Flat buffers whose parts are the tensors, each on a boundary of 256 values (as an allocator gives them)."""
    at, parts = 0, []
    for shape in shapes(c):
        n = math.prod(shape)
        parts.append((at, n, shape))
        at += _up(n, STATES)

    def tensors(flat):
        return [flat[a:a + n].view(shape) for a, n, shape in parts]

    inside = torch.zeros(at, device="cuda")
    for v in tensors(inside):
        v.fill_(1.0)
    gdt = DTYPES[c["grads"]]
    size = torch.exp(r.normal((at // STATES, 1), std=1.0)) * 1e-3
    s["p"] = r.normal((at,), std=0.02) * inside
    s["g"] = ((r.normal((at // STATES, STATES)) * size).view(-1) * inside).to(gdt)
    m = (r.normal((at // STATES, STATES)) * size * 0.3).view(-1) * inside
    root = (torch.exp(r.normal((at // STATES, STATES), std=0.5)) * size).view(-1) * inside
    if c["bits"] == 32:
        s["m"], s["v"] = m, root * root
    else:
        for name, t in (("m", m), ("v", root)):
            b = t.view(-1, STATES)
            s[name + "_scale"] = b.abs().amax(1) / TOP
            q = torch.where(s[name + "_scale"].unsqueeze(1) > 0, b / s[name + "_scale"].unsqueeze(1), 0.0)
            s[name] = (torch.clamp(q, min=2.0 ** -9) * (b > 0) if name == "v" else q).to(E4M3).view(-1)
        for name in ("m_scale", "v_scale"):
            s[name + "s"] = [s[name][a // STATES:a // STATES + -(-n // STATES)] for a, n, _ in parts]
    for name in ("p", "g", "m", "v"):
        s[name + "s"] = tensors(s[name])
    s["clip"] = torch.full((), 0.37, device="cuda") if c["clip"] else None
    s["hyper"] = dict(lr=3e-4, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)


# --------------------------------------------------------------------------
# the plain forms
# --------------------------------------------------------------------------

def _blocks(x, tile):
    """x [rows, cols] filled up with zeros, as [row blocks, rows, col blocks, cols]."""
    rows = BLOCK if tile else 1
    x = torch.nn.functional.pad(x, (0, -x.shape[1] % BLOCK, 0, -x.shape[0] % rows))
    return x.view(x.shape[0] // rows, rows, -1, BLOCK)


def _spread(scale, x, tile):
    """Each value's scale, [rows, cols] as x."""
    s = scale.repeat_interleave(BLOCK, 1)[:, :x.shape[1]]
    return s.repeat_interleave(BLOCK, 0)[:x.shape[0]] if tile else s


def _quantise(x, tile):
    """8-bit values and their scales: the least power of two that brings a block's largest to 448 or less."""
    x = x.float()
    m, e = torch.frexp(_blocks(x, tile).abs().amax((1, 3)))   # m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.clamp(e - 9 + (m > 0.875).to(e.dtype), min=-118)
    scale = ((e + 127) << 23).view(torch.float32)             # 2^e by its bits
    return (x / _spread(scale, x, tile)).to(E4M3), scale


def _values(q, scale, tile):
    return q.float() * _spread(scale, q, tile)


def plain_quant(s):
    c = s["case"]
    q, scale = _quantise(s["x"], c["tile"])
    if not c["both"]:
        return q, scale
    return (q, scale) + _quantise(s["x"].t(), c["tile"])


def plain_matmul(s):
    c = s["case"]
    y = _values(s["a"], s["a_scale"], False) @ _values(s["b"], s["b_scale"], c["tile"]).t()
    return y.to(DTYPES[c["out"]])


def plain_proj(s):
    x = _values(*_quantise(s["x"], False), False)
    return (x @ _values(s["w"], s["w_scale"], True).t()).to(s["x"].dtype)


def plain_proj_train(s):
    dt = s["x"].dtype
    w = _values(*_quantise(s["weight"], True), True)
    y = _values(*_quantise(s["x"], False), False) @ w.t()
    dx = _values(*_quantise(s["dy"], False), False) @ w
    xt, dyt = (_values(*_quantise(t.t(), False), False) for t in (s["x"], s["dy"]))
    return {"y": y.to(dt), "dx": dx.to(dt), "dweight": dyt @ xt.t()}


def _states_quantised(b, root):
    """Blocks of a state [n, 256] in 8 bits, and their scales; a root above zero stays above it."""
    a = b.abs().amax(1, keepdim=True)
    some, top = a > LEAST, torch.full_like(a, TOP)  # (a quotient with a number is a product with its inverse)
    q = (b * torch.where(some, top / a, 0.0)).to(E4M3)
    if root:
        q = torch.where((b > 0) & some & (q.float() == 0), torch.full_like(b, 2.0 ** -9), q.float()).to(E4M3)
    return q, torch.where(some, a / top, 0.0)[:, 0]


def plain_adamw(s):
    c, h = s["case"], s["hyper"]
    (b1, b2), t = h["betas"], c["step"]
    g = s["g"].float()
    if s["clip"] is not None:
        g = g * s["clip"]
    if c["bits"] == 32:
        m, v = s["m"], s["v"]
    else:
        m = (s["m"].float().view(-1, STATES) * s["m_scale"].unsqueeze(1)).view(-1)
        v = (s["v"].float().view(-1, STATES) * s["v_scale"].unsqueeze(1)).view(-1)
        v = v * v
    m = m * b1 + g * (1.0 - b1)
    v = v * b2 + (g * g) * (1.0 - b2)
    root = torch.sqrt(v)
    denominator = root * (1.0 / math.sqrt(1.0 - b2 ** t)) + h["eps"]
    s["p"].copy_(s["p"] * (1.0 - h["lr"] * h["weight_decay"]) - (m / denominator) * (h["lr"] / (1.0 - b1 ** t)))
    if c["bits"] == 32:
        s["m"].copy_(m)
        s["v"].copy_(v)
        return s["p"], s["m"], s["v"]
    for name, x in (("m", m), ("v", root)):
        q, scale = _states_quantised(x.view(-1, STATES), name == "v")
        s[name].copy_(q.view(-1))
        s[name + "_scale"].copy_(scale)
    return s["p"], s["m"], s["m_scale"], s["v"], s["v_scale"]


PLAIN = {"quant": plain_quant, "matmul": plain_matmul, "proj": plain_proj, "proj_train": plain_proj_train,
         "adamw": plain_adamw}


# --------------------------------------------------------------------------
# the framework's calls
# --------------------------------------------------------------------------

def run(state):
    s, c = state, state["case"]
    if not own:
        return PLAIN[c["op"]](s)
    import state_space_sequence_cumsum_gb300 as ssd
    if c["op"] == "quant":
        out = ssd.ssd_block_quantize(s["x"], tile=c["tile"], want_t=c["both"])
        return out if c["both"] else out[:2]
    if c["op"] == "matmul":
        return ssd.ssd_block_matmul(s["a"], s["a_scale"], s["b"], s["b_scale"], out_dtype=DTYPES[c["out"]])
    if c["op"] == "proj":
        return ssd.ssd_projection(s["x"], s["w"], s["w_scale"])[0]
    if c["op"] == "proj_train":
        w, w_scale, w_t, w_t_scale = ssd.ssd_block_quantize(s["weight"], tile=True, want_t=True)
        y, x_t, x_t_scale = ssd.ssd_projection(s["x"], w, w_scale, return_kept=True)
        g = ssd.ssd_projection_bwd(s["dy"], w_t, w_t_scale, x_t, x_t_scale)
        return {"y": y, "dx": g["dx"], "dweight": g["dweight"]}
    if c["bits"] == 32:
        ssd.ssd_adamw_step(s["ps"], s["gs"], s["ms"], s["vs"], c["step"], grad_scale=s["clip"], **s["hyper"])
        return s["p"], s["m"], s["v"]
    ssd.ssd_adamw_step(s["ps"], s["gs"], s["ms"], s["vs"], c["step"], m_scales=s["m_scales"],
                       v_scales=s["v_scales"], grad_scale=s["clip"], **s["hyper"])
    return s["p"], s["m"], s["m_scale"], s["v"], s["v_scale"]


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "quant":
        n, e = c["rows"] * c["cols"], 2 if c["dtype"] == "bf16" else 4
        ways = 2 if c["both"] else 1
        return {"bytes": n * (e + ways) + ways * 4 * n // (BLOCK * BLOCK if c["tile"] else BLOCK), "flops": 3 * n}
    if c["op"] == "matmul":
        m, n, k = c["m"], c["n"], c["k"]
        scales = 4 * (m * k // BLOCK + n * k // (BLOCK * BLOCK if c["tile"] else BLOCK))
        return {"bytes": (m + n) * k + scales + m * n * (2 if c["out"] == "bf16" else 4), "flops": 2 * m * n * k}
    if c["op"] in ("proj", "proj_train"):
        m, k, n, e = c["tokens"], c["inputs"], c["outputs"], 2 if c["dtype"] == "bf16" else 4
        if c["op"] == "proj":
            return {"bytes": m * (k + n) * e + n * k, "flops": 2 * m * n * k}
        return {"bytes": 2 * m * (k + n) * e + 8 * n * k, "flops": 6 * m * n * k}
    n = sum(math.prod(shape) for shape in shapes(c))
    return {"bytes": n * (8 + (2 if c["grads"] == "bf16" else 4) + (16 if c["bits"] == 32 else 4)), "flops": 16 * n}


# --------------------------------------------------------------------------
# 64 bits, from the definitions
# --------------------------------------------------------------------------

def _rounded(t):
    """64-bit values to the nearest e4m3 value (ties to an even last bit), as 64-bit values."""
    step = torch.exp2(torch.clamp(torch.floor(torch.log2(torch.clamp(t.abs(), min=2.0 ** -20))), min=-6.0) - 3.0)
    return torch.clamp(torch.round(t / step) * step, -TOP, TOP)


def _exact_scale(a):
    """The least power of two, 2^-118 or more, with a / scale at most 448."""
    e = torch.ceil(torch.log2(torch.clamp(a, min=2.0 ** -120) / TOP))
    e = torch.where(torch.exp2(e - 1.0) * TOP >= a, e - 1.0, e)
    e = torch.where(torch.exp2(e) * TOP < a, e + 1.0, e)
    return torch.exp2(torch.clamp(e, min=-118.0))


def _exact_quantise(x, tile):
    """(8-bit values, scales, what they stand for), column block by column block."""
    q, values, scales = torch.empty_like(x), torch.empty_like(x), []
    for j in range(0, x.shape[1], BLOCK):
        part = x[:, j:j + BLOCK]
        a = part.abs().amax(1)
        if tile:
            a = torch.stack([v.max() for v in a.split(BLOCK)])
        scale = _exact_scale(a)
        scales.append(scale)
        each = (scale.repeat_interleave(BLOCK)[:x.shape[0]] if tile else scale).unsqueeze(1)
        q[:, j:j + BLOCK] = _rounded(part / each)
        values[:, j:j + BLOCK] = q[:, j:j + BLOCK] * each
    return q, torch.stack(scales, 1), values


def _exact_values(q, scale, tile):
    values = q.double()
    for j in range(scale.shape[1]):
        each = scale[:, j].double()
        each = each.repeat_interleave(BLOCK)[:q.shape[0]] if tile else each
        values[:, j * BLOCK:(j + 1) * BLOCK] *= each.unsqueeze(1)
    return values


def _exact_states(x, root):
    b = x.view(-1, STATES)
    a = b.abs().amax(1, keepdim=True)
    some = a > LEAST
    q = _rounded(torch.where(some, b * TOP / torch.where(some, a, 1.0), 0.0))
    if root:
        q = torch.where((b > 0) & some, torch.clamp(q, min=2.0 ** -9), q)
    return q.view(-1), torch.where(some, a / TOP, 0.0)[:, 0]


def exact(case, seed):
    """The definitions in 64 bits."""
    c = case
    if work(c)["flops"] > 4e12 and c["op"] != "adamw":  # some 20 s of 64-bit products, and their memory
        return None
    s = prepare(c, seed)
    if c["op"] == "quant":
        x = s["x"].double()
        out = _exact_quantise(x, c["tile"])[:2]
        return out + _exact_quantise(x.t().contiguous(), c["tile"])[:2] if c["both"] else out
    if c["op"] == "matmul":
        return _exact_values(s["a"], s["a_scale"], False) @ _exact_values(s["b"], s["b_scale"], c["tile"]).t()
    if c["op"] == "proj":
        return _exact_quantise(s["x"].double(), False)[2] @ _exact_values(s["w"], s["w_scale"], True).t()
    if c["op"] == "proj_train":
        x, dy, w = s["x"].double(), s["dy"].double(), _exact_quantise(s["weight"].double(), True)[2]
        xt, dyt = (_exact_quantise(t.t().contiguous(), False)[2] for t in (x, dy))
        return {"y": _exact_quantise(x, False)[2] @ w.t(), "dx": _exact_quantise(dy, False)[2] @ w,
                "dweight": dyt @ xt.t()}
    h, t = s["hyper"], c["step"]
    (b1, b2), p, g = h["betas"], s["p"].double(), s["g"].double()
    if s["clip"] is not None:
        g = g * float(s["clip"])
    if c["bits"] == 32:
        m, v = s["m"].double(), s["v"].double()
    else:
        m = s["m"].double() * s["m_scale"].double().repeat_interleave(STATES)
        v = torch.square(s["v"].double() * s["v_scale"].double().repeat_interleave(STATES))
    m = torch.lerp(g, m, b1)
    v = torch.lerp(torch.square(g), v, b2)
    hat_m, hat_v = m / (1.0 - b1 ** t), v / (1.0 - b2 ** t)
    p = p - h["lr"] * (hat_m / (torch.sqrt(hat_v) + h["eps"]) + h["weight_decay"] * p)
    if c["bits"] == 32:
        return p, m, v
    return (p,) + _exact_states(m, False) + _exact_states(torch.sqrt(v), True)
