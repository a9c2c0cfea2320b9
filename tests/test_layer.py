"""GPU tests of the layer operators (convolution, selective scan, block norm)
against their float64 references, at the sizes and layouts where they can go
wrong.

Tolerances.  All arithmetic is f32 on exactly widened inputs, so an f32 result
carries a few units of 2^-24 per operation; fast exponentials and divisions
add up to about 2^-21.  A state's decays each carry the exponential's 2^-22,
and at most min(L, memory) <= 600 of them multiply up in the sizes below, so
600 * 2^-22 = 1.5e-4 of the result's scale bounds the scan in f32, and 2e-5
bounds the operators without a recurrence.  Sums over tokens add n terms in
f32, which stays under the same bounds relative to the sum's rms at these
sizes.  A bf16 result adds its rounding, 2^-9 of each element (2^-8 allowed)."""
import numpy as np
import pytest
import torch

from oracle import layer
import state_space_sequence_cumsum_gb300 as ssd

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
PLAIN, SCAN = 2e-5, 1.5e-4


def close(got, want, tol):
    g = got.detach().to("cpu", torch.float64).numpy()
    assert g.shape == want.shape
    assert np.array_equal(np.isnan(g), np.isnan(want))
    ok = np.isfinite(want)
    assert np.array_equal(ok, np.isfinite(g))
    if not ok.any():
        return
    g, w = g[ok], want[ok]
    rms = float(np.sqrt(np.mean(w * w)))
    bound = tol * (np.abs(w) + rms)
    if got.dtype == BF16:
        bound = bound + 2.0 ** -8 * np.abs(w)
    assert np.max(np.abs(g - w) - bound) <= 0.0


class Draw:
    def __init__(self, seed):
        self.g = torch.Generator().manual_seed(seed)

    def __call__(self, *shape, dtype=F32, std=1.0, mean=0.0):
        return (torch.randn(shape, generator=self.g) * std + mean).to(dtype)


def cu(t):
    return None if t is None else t.cuda()


def sliced(t, extra, offset):
    """The same values as a slice of a wider tensor on the GPU."""
    wide = torch.full(t.shape[:-1] + (t.shape[-1] + extra,), float("nan"), dtype=t.dtype, device="cuda")
    v = wide[..., offset:offset + t.shape[-1]]
    v.copy_(t)
    return v


# ------------------------------------------------------------- convolution

CONV = [  # batch, seqlen, dim, width, dtype, silu, bias, carry, (extra, offset) of x's rows
    (2, 37, 64, 4, BF16, True, True, False, None),
    (2, 37, 64, 4, BF16, True, True, True, (64, 8)),
    (1, 1, 8, 4, F32, True, True, True, None),          # one token: the state mixes old and new
    (3, 2, 40, 4, BF16, True, False, True, None),       # fewer tokens than the window
    (1, 600, 33, 3, F32, True, True, True, (5, 3)),     # odd channels, unaligned rows
    (2, 301, 24, 2, BF16, False, True, False, (3, 1)),
    (5, 130, 260, 3, F32, False, False, False, None),
    (1, 5000, 16, 4, BF16, True, True, True, None),     # few channels, many tokens
]


def conv_inputs(case, seed=0):
    b, L, D, W, dt, silu, bias, carry, rows = case
    r = Draw(seed)
    x = r(b, L, D, dtype=dt)
    return (x, sliced(x, *rows) if rows else x.cuda(), r(D, W, std=0.5), r(D) if bias else None,
            r(b, W - 1, D, dtype=dt) if carry else None, "silu" if silu else None, r)


@pytest.mark.parametrize("case", CONV)
def test_conv(case):
    x, xd, w, bias, init, act, _ = conv_inputs(case)
    y, fin = ssd.ssd_causal_conv(xd, w.cuda(), cu(bias), act, cu(init), return_final_state=True)
    wy, wf = layer.conv(x, w, bias, init, act is not None)
    close(y, wy, PLAIN)
    assert np.array_equal(fin.cpu().double().numpy(), wf)  # carried tokens are copies


@pytest.mark.parametrize("case", CONV)
@pytest.mark.parametrize("with_dfinal", [False, True])
def test_conv_bwd(case, with_dfinal):
    x, xd, w, bias, init, act, r = conv_inputs(case, 1)
    dy = r(*x.shape, dtype=x.dtype)
    df = r(x.shape[0], w.shape[1] - 1, x.shape[2], dtype=x.dtype) if with_dfinal else None
    g = ssd.ssd_causal_conv_bwd(xd, w.cuda(), dy.cuda(), cu(bias), act, cu(init), cu(df))
    want = layer.conv_bwd(x, w, dy, bias, init, df, act is not None)
    assert (g["dbias"] is None) == (bias is None)
    for k, v in g.items():
        if v is not None:
            close(v, want[k], PLAIN)


# Two-byte rows off vector boundaries, 64 channels and more: channels a warp
# apart, the last warp's shared with its neighbour.
CONV_ODD = [
    (1, 1, 65, 4, BF16, True, True, True, None),
    (2, 19, 64, 3, BF16, True, True, True, (7, 3)),
    (2, 70, 127, 2, BF16, True, False, False, None),
    (3, 133, 193, 4, BF16, False, True, True, (8, 5)),
    (2, 1030, 131, 4, BF16, True, True, True, (4, 1)),
]


@pytest.mark.parametrize("case", CONV_ODD)
def test_conv_off_boundaries(case):
    test_conv(case)
    test_conv_bwd(case, True)


@pytest.mark.parametrize("b,D,W,dt,rows", [(1, 8, 4, F32, None), (7, 260, 3, BF16, (12, 4)), (130, 33, 2, BF16, None),
                                           (3, 5, 4, F32, (2, 1))])
def test_conv_step_continues_a_prompt(b, D, W, dt, rows):
    r = Draw(2)
    x, w, bias = r(b, 9, D, dtype=dt), r(D, W, std=0.5).cuda(), r(D).cuda()
    full, last = ssd.ssd_causal_conv(x.cuda(), w, bias, return_final_state=True)
    y0, state = ssd.ssd_causal_conv(x[:, :6].contiguous().cuda(), w, bias, return_final_state=True)
    for t in range(6, 9):
        xt = sliced(x[:, t], *rows) if rows else x[:, t].contiguous().cuda()
        if t == 7:  # out of place, then in place
            y, state = ssd.ssd_causal_conv_step(xt, w, state, bias, state_out=torch.empty_like(state))
        else:
            y, state = ssd.ssd_causal_conv_step(xt, w, state, bias)
        assert torch.equal(y, full[:, t])
    assert torch.equal(state, last)


def test_conv_without_tokens():
    init = Draw(3)(2, 3, 16).cuda()
    w = torch.ones(16, 4, device="cuda")
    y, fin = ssd.ssd_causal_conv(torch.empty(2, 0, 16, device="cuda"), w, initial_state=init,
                                 return_final_state=True)
    assert y.shape == (2, 0, 16) and torch.equal(fin, init)
    df = Draw(4)(2, 3, 16).cuda()
    g = ssd.ssd_causal_conv_bwd(torch.empty(2, 0, 16, device="cuda"), w, torch.empty(2, 0, 16, device="cuda"),
                                initial_state=init, dfinal=df)
    assert torch.equal(g["dinit"], df) and float(g["dweight"].abs().max()) == 0.0


def test_conv_infinities_stay_in_their_window():
    """An infinite input reaches its W outputs and no others."""
    x = Draw(5)(1, 20, 8)
    x[0, 7, 2] = float("inf")
    w, dy = Draw(6)(8, 4, std=0.5), Draw(7)(1, 20, 8)
    y, _ = ssd.ssd_causal_conv(x.cuda(), w.cuda(), activation=None)
    close(y, layer.conv(x, w, silu=False)[0], PLAIN)
    g = ssd.ssd_causal_conv_bwd(x.cuda(), w.cuda(), dy.cuda(), activation=None)
    close(g["dx"], layer.conv_bwd(x, w, dy, silu=False)["dx"], PLAIN)


# ---------------------------------------------------------- selective scan

SCANS = [  # batch, seqlen, dim, N, groups, dtype, gated, skip, bias, softplus, carry, rows
    (2, 37, 64, 16, 1, BF16, True, True, True, True, False, None),
    (2, 50, 96, 16, 1, F32, True, True, True, True, True, None),
    (1, 1, 8, 16, 1, F32, True, True, True, True, True, None),           # one token
    (1, 16, 40, 16, 1, BF16, False, True, True, True, True, (64, 8)),    # exactly one chunk
    (3, 17, 36, 4, 3, F32, True, False, True, True, True, None),         # a chunk and one token, groups
    (1, 333, 20, 5, 2, F32, True, True, False, True, True, (3, 1)),      # odd states, unaligned rows
    (2, 130, 10, 1, 1, BF16, False, False, False, False, False, None),   # no softplus: dt given positive
    (1, 600, 32, 64, 1, BF16, True, True, True, True, True, None),
    (2, 90, 24, 32, 2, F32, False, True, True, True, False, None),
    (1, 500, 7, 8, 1, F32, True, True, True, True, True, None),          # dim not a multiple of four
    (1, 70, 650, 16, 1, BF16, True, True, True, True, True, None),       # several channel blocks, ragged
    (1, 40, 1300, 3, 2, F32, True, True, True, True, True, None),
    (1, 600, 16, 16, 1, F32, True, True, True, True, True, None),        # segments
]


def scan_inputs(case, seed=0):
    b, L, D, N, G, dt, gated, skip, bias, softplus, carry, rows = case
    r = Draw(seed)
    t = {"u": r(b, L, D, dtype=dt), "dt": r(b, L, D, dtype=dt, std=0.5)}
    if not softplus:
        t["dt"] = (t["dt"].float().abs() * 0.1).to(dt)
    t["A"] = -torch.exp(torch.rand(D, N, generator=r.g) * 2.77)
    t["B"], t["C"] = r(b, L, G, N, dtype=dt), r(b, L, G, N, dtype=dt)
    t["D"] = r(D) if skip else None
    t["z"] = r(b, L, D, dtype=dt) if gated else None
    t["dt_bias"] = r(D, std=0.5, mean=-4.0) if bias else None
    t["init"] = r(b, D, N) if carry else None
    d = {k: cu(v) for k, v in t.items()}
    if rows:
        for k in ("u", "dt", "z"):
            if t[k] is not None:
                d[k] = sliced(t[k], *rows)
        for k in ("B", "C"):
            d[k] = sliced(t[k].flatten(2), *rows).unflatten(2, (G, N))
    return t, d, softplus, r


def ref_scan(t, softplus):
    return layer.scan(t["u"], t["dt"], t["A"], t["B"], t["C"], t["D"], t["z"], t["dt_bias"], softplus, t["init"])


@pytest.mark.parametrize("case", SCANS)
def test_scan(case):
    t, d, sp, _ = scan_inputs(case)
    y, fin, kept = ssd.ssd_selective_scan(d["u"], d["dt"], d["A"], d["B"], d["C"], d["D"], d["z"], d["dt_bias"],
                                          sp, d["init"], return_chunk_states=True)
    wy, h = ref_scan(t, sp)
    close(y, wy, SCAN)
    close(fin, h[:, -1], SCAN)
    T = ssd.ssd_selective_scan_chunk()
    close(kept, h[:, 0:t["u"].shape[1]:T], SCAN)


@pytest.mark.parametrize("case", SCANS)
@pytest.mark.parametrize("keep,with_dfinal", [(True, True), (False, False)])
def test_scan_bwd(case, keep, with_dfinal):
    t, d, sp, r = scan_inputs(case, 1)
    dy = r(*t["u"].shape, dtype=t["u"].dtype)
    df = r(t["u"].shape[0], *t["A"].shape) if with_dfinal else None
    args = (d["u"], d["dt"], d["A"], d["B"], d["C"], d["D"])
    kept = None
    if keep:
        kept = ssd.ssd_selective_scan(*args, d["z"], d["dt_bias"], sp, d["init"], return_chunk_states=True)[2]
    g = ssd.ssd_selective_scan_bwd(*args, dy.cuda(), d["z"], d["dt_bias"], sp, d["init"], cu(df), kept)
    want = layer.scan_bwd(t["u"], t["dt"], t["A"], t["B"], t["C"], dy, t["D"], t["z"], t["dt_bias"], sp, t["init"], df)
    for name, inp in (("dD", "D"), ("dz", "z"), ("ddt_bias", "dt_bias")):
        assert (g[name] is None) == (t[inp] is None)
    for k, v in g.items():
        if v is not None:
            close(v, want[k], 2 * SCAN)  # two recurrences, forward and reverse


@pytest.mark.parametrize("case", [c for c in SCANS if c[1] > 1])
def test_scan_step_continues_a_prompt(case):
    t, d, sp, _ = scan_inputs(case, 2)
    cut = t["u"].shape[1] - min(3, t["u"].shape[1] - 1)
    wy, h = ref_scan(t, sp)

    def part(k, lo, hi):
        return None if d[k] is None else d[k][:, lo:hi]
    first = [part(k, 0, cut) for k in ("u", "dt", "B", "C", "z")]
    first = [None if v is None else v.contiguous() for v in first]
    _, state, _ = ssd.ssd_selective_scan(first[0], first[1], d["A"], first[2], first[3], d["D"], first[4],
                                         d["dt_bias"], sp, d["init"])
    for i in range(cut, t["u"].shape[1]):
        out = None if i % 2 else torch.empty_like(state)
        y, state = ssd.ssd_selective_scan_step(d["u"][:, i], d["dt"][:, i], d["A"], d["B"][:, i], d["C"][:, i],
                                               d["D"], state, None if d["z"] is None else d["z"][:, i],
                                               d["dt_bias"], sp, state_out=out)
        close(y, wy[:, i], SCAN)
    close(state, h[:, -1], SCAN)


def test_scan_without_tokens():
    r = Draw(8)
    A, init, df = -torch.ones(8, 16).cuda(), r(2, 8, 16).cuda(), r(2, 8, 16).cuda()
    e = torch.empty(2, 0, 8, device="cuda")
    m = torch.empty(2, 0, 16, device="cuda")
    y, fin, kept = ssd.ssd_selective_scan(e, e, A, m, m, initial_state=init, return_chunk_states=True)
    assert y.shape == (2, 0, 8) and kept.shape == (2, 0, 8, 16) and torch.equal(fin, init)
    g = ssd.ssd_selective_scan_bwd(e, e, A, m, m, None, e, initial_state=init, dfinal=df, chunk_states=kept)
    assert torch.equal(g["dinit"], df) and float(g["dA"].abs().max()) == 0.0 and g["dB"].shape == m.shape


@pytest.mark.parametrize("L", [40, 600])
def test_scan_state_carried_in_place_and_prompt_cut(L):
    """A prompt in two calls, the second updating the first's state in place."""
    t, d, sp, _ = scan_inputs((1, L, 48, 16, 1, F32, True, True, True, True, True, None), 3)
    wy, h = ref_scan(t, sp)
    cut = L // 2 + 3
    state = d["init"].clone()
    ys = []
    for lo, hi in ((0, cut), (cut, L)):
        p = {k: d[k][:, lo:hi].contiguous() for k in ("u", "dt", "B", "C", "z")}
        y, out, _ = ssd.ssd_selective_scan(p["u"], p["dt"], d["A"], p["B"], p["C"], d["D"], p["z"], d["dt_bias"], sp,
                                           state, final_state=state)
        assert out.data_ptr() == state.data_ptr()
        ys.append(y)
    close(torch.cat(ys, 1), wy, SCAN)
    close(state, h[:, -1], SCAN)


def test_scan_large_and_tiny_steps():
    """Raw steps from -60 to 60: softplus underflows to a full carry and grows
    to a full reset of the state, without inf or NaN."""
    case = (1, 64, 12, 16, 1, F32, True, True, False, True, True, None)
    t, d, sp, r = scan_inputs(case, 4)
    t["dt"] = torch.linspace(-60, 60, 64 * 12).reshape(1, 64, 12)
    d["dt"] = t["dt"].cuda()
    y, fin, kept = ssd.ssd_selective_scan(d["u"], d["dt"], d["A"], d["B"], d["C"], d["D"], d["z"],
                                          initial_state=d["init"], return_chunk_states=True)
    wy, h = ref_scan(t, True)
    close(y, wy, SCAN)
    close(fin, h[:, -1], SCAN)
    dy = r(1, 64, 12)
    g = ssd.ssd_selective_scan_bwd(d["u"], d["dt"], d["A"], d["B"], d["C"], d["D"], dy.cuda(), d["z"],
                                   initial_state=d["init"], chunk_states=kept)
    want = layer.scan_bwd(t["u"], t["dt"], t["A"], t["B"], t["C"], dy, t["D"], t["z"], None, True, t["init"])
    for k, v in g.items():
        if v is not None:
            close(v, want[k], 2 * SCAN)


# -------------------------------------------------------------- block norm

NORMS = [  # tokens, dim, dtype, residual dtype (None: no residual), post, gate rows
    (5, 64, BF16, F32, True, 5),
    (12, 2560, BF16, F32, True, 4),
    (12, 2560, BF16, BF16, True, 0),
    (700, 96, F32, F32, True, 1),
    (7, 33, F32, F32, False, 7),
    (9, 1001, BF16, F32, True, 3),       # single channels
    (1, 1, F32, F32, True, 1),
    (3, 4100, BF16, BF16, False, 0),
    (6, 9000, F32, F32, True, 2),        # more vectors a thread
    (2, 32768, BF16, F32, True, 1),
    (3, 2563, BF16, None, True, 0),
    (1300, 128, BF16, F32, True, 650),   # gate rows of two tokens
]


def norm_inputs(case, seed=0):
    T, D, dt, rdt, post, rows = case
    r = Draw(seed)
    return (r(T, D, dtype=dt), None if rdt is None else r(T, D, dtype=rdt, std=2.0), r(D, std=0.3, mean=1.0),
            r(D, std=0.3, mean=1.0) if post else None, r(rows, D) if rows else None, r)


@pytest.mark.parametrize("case", NORMS)
def test_block_norm(case):
    y, res, w, pw, gate, _ = norm_inputs(case)
    out, rr = ssd.ssd_block_norm(cu(y), cu(res), cu(w), cu(pw), cu(gate), 0.3, 1e-5)
    wo, wr = layer.block_norm(y, res, w, pw, gate, 0.3, 1e-5)
    close(out, wo, PLAIN)
    close(rr, wr, PLAIN)
    assert rr.dtype == (res.dtype if res is not None else y.dtype)


@pytest.mark.parametrize("case", NORMS)
@pytest.mark.parametrize("with_dr", [True, False])
def test_block_norm_bwd(case, with_dr):
    y, res, w, pw, gate, r = norm_inputs(case, 1)
    res = r(*y.shape, dtype=y.dtype) if res is None else res  # the residual after the block
    dout = r(*y.shape, dtype=y.dtype)
    dr = r(*y.shape, dtype=res.dtype) if with_dr else None
    g = ssd.ssd_block_norm_bwd(cu(y), cu(res), cu(w), cu(dout), cu(dr), cu(pw), cu(gate), 0.3, 1e-5)
    want = layer.block_norm_bwd(y, res, w, dout, dr, pw, gate, 0.3, 1e-5)
    assert (g["dgate"] is None) == (gate is None) and (g["dpost_weight"] is None) == (pw is None)
    for k, v in g.items():
        if v is not None:
            close(v, want[k], PLAIN)


def test_block_norm_in_place_and_leading_dimensions():
    r = Draw(2)
    y, res, w, gate = r(2, 7, 48), r(2, 7, 48), r(48), r(2, 1, 48)
    wo, wr = layer.block_norm(y.reshape(14, 48), res.reshape(14, 48), w, None, gate.reshape(2, 48))
    rd = res.cuda()
    out, rr = ssd.ssd_block_norm(y.cuda(), rd, w.cuda(), gate=gate.cuda(), residual_out=rd)
    assert rr.data_ptr() == rd.data_ptr() and out.shape == y.shape
    close(out.reshape(14, 48), wo, PLAIN)
    close(rd.reshape(14, 48), wr, PLAIN)


def test_block_norm_zero_rows_and_no_tokens():
    z = torch.zeros(3, 40, device="cuda")
    w = torch.ones(40, device="cuda")
    out, rr = ssd.ssd_block_norm(z, z, w, w, eps=1e-5)
    assert float(out.abs().max()) == 0.0 and float(rr.abs().max()) == 0.0
    g = ssd.ssd_block_norm_bwd(z, z, w, torch.ones_like(z), None, w)
    assert bool(torch.isfinite(g["dy"]).all()) and bool(torch.isfinite(g["dresidual"]).all())
    e = torch.empty(0, 40, device="cuda")
    out, rr = ssd.ssd_block_norm(e, e, w)
    assert out.shape == (0, 40)
    g = ssd.ssd_block_norm_bwd(e, e, w, e, None, w, gate=None)
    assert float(g["dweight"].abs().max()) == 0.0 and float(g["dpost_weight"].abs().max()) == 0.0


# ------------------------------------------------- shared: autograd, streams

def directional(loss, tensors, grads, tol):
    """Central difference along a random direction of all inputs together.
    With step h = 2^-7 the truncation error is h^2 / 6 times the third
    derivative and the f32 rounding of the loss about 2^-22 |loss| / h; tol
    covers both, relative to the sum of the products' magnitudes."""
    g = torch.Generator(device="cuda").manual_seed(9)
    dirs = [torch.randn(t.shape, generator=g, device="cuda") for t in tensors]
    h = 2.0 ** -7
    up = loss([t + h * d for t, d in zip(tensors, dirs)])
    down = loss([t - h * d for t, d in zip(tensors, dirs)])
    got = sum(float((a.double() * d.double()).sum()) for a, d in zip(grads, dirs))
    size = sum(float((a.double() * d.double()).norm()) for a, d in zip(grads, dirs))
    assert abs((up - down) / (2 * h) - got) <= tol * size


def test_gradients_against_differences():
    r = Draw(10)
    B, L, D, N = 2, 24, 16, 8
    x, w, b, init = (r(B, L, D).cuda(), r(D, 4, std=0.5).cuda(), r(D).cuda(), r(B, 3, D).cuda())
    dy, df = r(B, L, D).cuda(), r(B, 3, D).cuda()

    def conv_loss(t):
        y, fin = ssd.ssd_causal_conv(t[0], t[1], t[2], initial_state=t[3], return_final_state=True)
        return float((y.double() * dy).sum() + (fin.double() * df).sum())
    leaves = [t.requires_grad_(True) for t in (x, w, b, init)]
    y, fin = ssd.CausalConvFunction.apply(*leaves)
    torch.autograd.backward([y, fin], [dy, df])
    directional(conv_loss, [t.detach() for t in leaves], [t.grad for t in leaves], 1e-2)

    u, dt, z = (r(B, L, D).cuda() for _ in range(3))
    A, Bm, Cm = -torch.exp(r(D, N, std=0.3)).cuda(), r(B, L, N).cuda(), r(B, L, N).cuda()
    Dv, bias, h0, dh = r(D).cuda(), r(D, mean=-1.0).cuda(), r(B, D, N).cuda(), r(B, D, N).cuda()

    def scan_loss(t):
        y, fin, _ = ssd.ssd_selective_scan(*t[:6], z=t[6], dt_bias=t[7], initial_state=t[8])
        return float((y.double() * dy).sum() + (fin.double() * dh).sum())
    leaves = [t.requires_grad_(True) for t in (u, dt, A, Bm, Cm, Dv, z, bias, h0)]
    y, fin = ssd.SelectiveScanFunction.apply(*leaves)
    torch.autograd.backward([y, fin], [dy, dh])
    directional(scan_loss, [t.detach() for t in leaves], [t.grad for t in leaves], 1e-2)

    yb, res, wt, pw, gate = (r(B * L, D).cuda(), r(B * L, D).cuda(), r(D).cuda(), r(D).cuda(), r(B, D).cuda())
    dres = r(B * L, D).cuda()

    def norm_loss(t):
        out, rr = ssd.ssd_block_norm(*t, scale=0.5)
        return float((out.double() * dy.reshape(B * L, D)).sum() + (rr.double() * dres).sum())
    leaves = [t.requires_grad_(True) for t in (yb, res, wt, pw, gate)]
    out, rr = ssd.BlockNormFunction.apply(*leaves, 0.5)
    torch.autograd.backward([out, rr], [dy.reshape(B * L, D), dres])
    directional(norm_loss, [t.detach() for t in leaves], [t.grad for t in leaves], 1e-2)


def test_results_repeat_bit_for_bit_and_on_another_stream():
    t, d, sp, r = scan_inputs((2, 600, 96, 16, 1, BF16, True, True, True, True, True, None), 11)
    dy = r(*t["u"].shape, dtype=BF16).cuda()
    args = (d["u"], d["dt"], d["A"], d["B"], d["C"], d["D"])
    one = ssd.ssd_selective_scan_bwd(*args, dy, d["z"], d["dt_bias"], sp, d["init"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    two = ssd.ssd_selective_scan_bwd(*args, dy, d["z"], d["dt_bias"], sp, d["init"], stream=side)
    side.synchronize()
    for k in one:
        assert torch.equal(one[k], two[k])


def test_under_graph_capture():
    """All operators launch kernels only: a step captured in a graph replays."""
    t, d, sp, _ = scan_inputs((4, 1, 64, 16, 1, BF16, True, True, True, True, True, None), 12)
    w = Draw(13)(64, 4).cuda()
    cs = torch.zeros(4, 3, 64, dtype=BF16, device="cuda")
    s0 = d["init"].clone()
    u = d["u"][:, 0]

    def step():
        x, _ = ssd.ssd_causal_conv_step(u, w, cs)
        y, _ = ssd.ssd_selective_scan_step(x, d["dt"][:, 0], d["A"], d["B"][:, 0], d["C"][:, 0], d["D"], s0,
                                           d["z"][:, 0], d["dt_bias"])
        return ssd.ssd_block_norm(y, u.contiguous(), torch.ones(64, device="cuda"))[0]
    want = [step().clone() for _ in range(3)]
    cs.zero_()
    s0.copy_(d["init"])
    graph = torch.cuda.CUDAGraph()
    keep = cs.clone(), s0.clone()
    with torch.cuda.graph(graph):
        out = step()
    cs.copy_(keep[0])
    s0.copy_(keep[1])
    for k in range(3):
        graph.replay()
        assert torch.equal(out, want[k])
