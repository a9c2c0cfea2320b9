"""The optimiser's step on the GPU against the float64 definition.

Tolerances.  m and v are two products and a sum of f32 values (three roundings
of their terms: 2^-22 of the terms' magnitudes, with a gradient scale 2^-21).
The update is a quotient with a root in its denominator: seven roundings and two
approximations of an ulp or two, 2^-19 of its magnitude, beside one rounding of
p.  8-bit states: the value that is rounded is the definition's within 2^-20, so
a state is off by at most one step of the type where a border lies between, and
elsewhere by its scale's 2^-23."""
import numpy as np
import pytest
import torch

import state_space_sequence_cumsum_gb300 as ssd
from oracle import blocks

pytestmark = pytest.mark.gpu

BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
HYPER = dict(lr=1e-2, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
HALF_STEP = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def np64(t):
    return t.detach().float().double().cpu().numpy().reshape(-1)


def problem(sizes, bits, p_dtype=F32, g_dtype=F32, seed=0, zero_states=False):
    g = torch.Generator().manual_seed(seed)

    def rand(n, std=1.0):
        return torch.randn(n, generator=g) * std * torch.exp(torch.randn((-(-n // 64)), generator=g)).repeat_interleave(64)[:n]
    out = {k: [] for k in ("params", "grads", "m", "v", "m_scales", "v_scales")}
    for n in sizes:
        p, gr = rand(n).to(p_dtype), rand(n, 0.1).to(g_dtype)
        m, root = (rand(n, 0.03), rand(n, 0.1).abs()) if not zero_states else (torch.zeros(n), torch.zeros(n))
        out["params"].append(p.cuda())
        out["grads"].append(gr.cuda())
        if bits == 32:
            out["m"].append(m.cuda())
            out["v"].append((root * root).cuda())
        else:
            for name, t, is_root in (("m", m, False), ("v", root, True)):
                q, s = blocks.quantise_state(t.double().numpy(), is_root)
                out[name].append(torch.tensor(q).to(E4).cuda())
                out[name + "_scales"].append(torch.tensor(s).float().cuda())
    if bits == 32:
        del out["m_scales"], out["v_scales"]
    return out


def run(s, step=3, **kw):
    ssd.ssd_adamw_step(s["params"], s["grads"], s["m"], s["v"], step, m_scales=s.get("m_scales"),
                       v_scales=s.get("v_scales"), **{**HYPER, **kw})


def clones(s):
    return {k: [t.clone() for t in v] for k, v in s.items()}


def states_of(s, i):
    m, v = np64(s["m"][i]), np64(s["v"][i])
    if "m_scales" in s:
        m = blocks.state_values(m, np64(s["m_scales"][i]))
        v = blocks.state_values(v, np64(s["v_scales"][i])) ** 2
    return m, v


def check(before, after, step=3, grad_scale=1.0, **kw):
    h = {**HYPER, **kw}
    for i, p in enumerate(after["params"]):
        m0, v0 = states_of(before, i)
        p0, g = np64(before["params"][i]), np64(before["grads"][i])
        wp, wm, wv = blocks.adamw(p0, g, m0, v0, step, grad_scale=grad_scale, **h)
        b1, b2 = h["betas"]
        gs = np.abs(g * grad_scale)
        tol_m = 2.0 ** -21 * (b1 * np.abs(m0) + (1 - b1) * gs)
        tol_v = 2.0 ** -20 * (b2 * v0 + (1 - b2) * gs * gs) + 1e-44
        # m's own error goes into the update as a share of its terms
        root = np.sqrt(wv / (1 - b2 ** step)) + h["eps"]
        update = h["lr"] / (1 - b1 ** step) * (b1 * np.abs(m0) + (1 - b1) * gs) / root
        tol_p = 2.0 ** -19 * update + 2.0 ** -22 * np.abs(p0) + HALF_STEP[p.dtype] * np.abs(wp) * (1 + 2.0 ** -12)
        assert (np.abs(np64(p) - wp) <= tol_p).all()
        if "m_scales" not in after:
            assert (np.abs(np64(after["m"][i]) - wm) <= tol_m).all()
            assert (np.abs(np64(after["v"][i]) - wv) <= tol_v).all()
            continue
        for name, want, is_root in (("m", wm, False), ("v", np.sqrt(wv), True)):
            q, s = blocks.quantise_state(want, is_root)
            got_q, got_s = np64(after[name][i]), np64(after[name + "_scales"][i])
            np.testing.assert_allclose(got_s, s, rtol=2.0 ** -19, atol=0)
            other = got_q != q
            assert other.sum() <= 1e-3 * other.size + 2
            step8 = np.ldexp(1.0, np.maximum(np.frexp(np.maximum(np.abs(q), np.abs(got_q)))[1] - 1, -6) - 3)
            assert (np.abs(got_q - q) <= step8).all()


SIZES = [[1], [256], [255, 257], [2048, 2049, 7, 0, 4096], [100000], [3, 5000, 33, 1] * 3]


@pytest.mark.parametrize("sizes", SIZES, ids=str)
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("p_dtype,g_dtype", [(F32, F32), (F32, BF), (BF, BF), (BF, F32)])
def test_step(sizes, bits, p_dtype, g_dtype):
    s = problem(sizes, bits, p_dtype, g_dtype)
    before = clones(s)
    run(s)
    check(before, s)
    assert all(torch.equal(a, b) for a, b in zip(before["grads"], s["grads"]))


@pytest.mark.parametrize("bits", [32, 8])
def test_more_tensors_than_one_launch_holds(bits):
    sizes = [(i * 37) % 700 for i in range(1100)]
    s = problem(sizes, bits)
    before = clones(s)
    run(s)
    check(before, s)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("kw", [dict(weight_decay=0.0), dict(betas=(0.0, 0.0)), dict(eps=1e-3, lr=0.5), dict(lr=0.0)], ids=str)
@pytest.mark.parametrize("step", [1, 2, 1000000])
def test_settings(bits, kw, step):
    s = problem([700, 20], bits, zero_states=step == 1)
    before = clones(s)
    run(s, step=step, **kw)
    check(before, s, step=step, **kw)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("device", [False, True])
def test_numbers_and_scalars_on_the_device(bits, device):
    """The same with the learning rate, the step and the gradients' factor given
    as numbers and as tensors."""
    s = problem([5000, 3], bits)
    before = clones(s)
    if device:
        run(s, step=torch.tensor(7, device="cuda"), lr=torch.tensor([0.02], device="cuda"),
            grad_scale=torch.tensor(0.25, device="cuda"))
    else:
        run(s, step=7, lr=0.02, grad_scale=0.25)
    check(before, s, step=7, grad_scale=0.25, lr=float(np.float32(0.02)))


@pytest.mark.parametrize("bits", [32, 8])
def test_unaligned_tensors_and_what_lies_beside_them(bits):
    """Parts of larger buffers off the vectors' boundaries; their neighbours stay."""
    s = problem([1000], bits)
    want = clones(s)
    run(want)
    bufs, parts = {}, {}
    for k, (t,) in s.items():
        buf = torch.full((t.numel() + 32,), 3.0, device="cuda").to(t.dtype)
        bufs[k] = buf
        parts[k] = [buf[5:5 + t.numel()]]
        parts[k][0].copy_(t)
    run(parts)
    for k in s:
        assert torch.equal(parts[k][0].float(), want[k][0].float())
        assert bool((bufs[k][:5].float() == 3).all()) and bool((bufs[k][5 + s[k][0].numel():].float() == 3).all())


def test_zeros_stay_zeros_and_nothing_is_divided_by_zero():
    for bits in (32, 8):
        s = problem([600], bits, zero_states=True)
        s["grads"][0].zero_()
        p0 = s["params"][0].clone()
        run(s, weight_decay=0.0, step=1)
        assert torch.equal(s["params"][0], p0) and not s["m"][0].float().any() and not s["v"][0].float().any()


def test_a_root_above_zero_is_kept_above_zero():
    """Gradients 10^5 below the block's largest: their averages of squares do not
    vanish, so their updates stay of the order of the learning rate."""
    s = problem([256], 8, zero_states=True)
    g = torch.full((256,), 1e-6, device="cuda")
    g[0] = 1.0
    s["grads"] = [g]
    p0 = s["params"][0].clone()
    for t in (1, 2):
        run(s, step=t, lr=1e-3, weight_decay=0.0)
    assert bool((s["v"][0].float() > 0).all())
    assert float((s["params"][0] - p0).abs().max()) <= 2.1e-3


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_what_is_not_finite_stays_in_its_block(bits, bad):
    s = problem([1024], bits)
    s["grads"][0][300] = bad
    run(s)
    touched = torch.zeros(1024, dtype=torch.bool)
    touched[256:512] = bits == 8
    touched[300] = True
    for name in ("m", "v"):
        t = s[name][0].float().cpu()
        if bits == 8:
            t = t * s[name + "_scales"][0].cpu().repeat_interleave(256)
            assert torch.equal(torch.isnan(t), touched)
        else:
            assert torch.equal(~torch.isfinite(t), touched)
    p = s["params"][0].cpu()
    assert bool(torch.isfinite(torch.cat([p[:300], p[301:]])).all())


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_and_replayed(bits):
    """Step, learning rate and gradients change between the replays."""
    s = problem([3000, 17], bits)
    want = clones(s)
    step, lr = torch.tensor(0, device="cuda"), torch.tensor(0.0, device="cuda")
    run(clones(s), step=torch.tensor(1, device="cuda"), lr=lr)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step += 1
        run(s, step=step, lr=lr)
    step.zero_()
    for t in range(1, 4):
        lr.fill_(0.01 * t)
        for g in s["grads"]:
            g.mul_(0.9)
        for g in want["grads"]:
            g.mul_(0.9)
        graph.replay()
        before = clones(want)
        run(want, step=torch.tensor(t, device="cuda"), lr=lr)
        check(before, want, step=t, lr=float(lr))
        for k in s:
            assert all(torch.equal(a.float(), b.float()) for a, b in zip(s[k], want[k]))


def test_streams():
    s = problem([5000, 9], 8)
    want = clones(s)
    run(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    run(s, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for k in s:
        assert all(torch.equal(a.float(), b.float()) for a, b in zip(s[k], want[k]))


def test_a_tensor_of_more_than_2_to_the_31_elements():
    n = (1 << 31) + 1027
    p = torch.zeros(n, dtype=BF, device="cuda")
    g = torch.ones(n, dtype=BF, device="cuda")
    m, v = (torch.zeros(n, dtype=torch.uint8, device="cuda").view(E4) for _ in range(2))
    ms, vs = (torch.zeros(-(-n // 256), device="cuda") for _ in range(2))
    g[-2] = -3.0
    ssd.ssd_adamw_step([p], [g], [m], [v], 1, m_scales=[ms], v_scales=[vs], lr=0.5, weight_decay=0.0)
    # the first step moves every element by the learning rate against its gradient
    assert float(p[-2]) == 0.5 and bool((p[:-2] == -0.5).all()) and float(p[-1]) == -0.5
    assert float(m[-2].float()) == -448.0 and bool((m[:1 << 31].view(torch.uint8) == m[0].view(torch.uint8)).all())


# ----------------------------------------------------------------- optimiser

@pytest.mark.parametrize("bits", [32, 8])
def test_optimiser_is_the_step(bits):
    """Groups, types and missing gradients; against torch's in 32 bits."""
    g = torch.Generator().manual_seed(1)
    shapes = [(30, 40), (7,), (300, 20), (11,)]
    first = [torch.randn(s, generator=g).cuda() for s in shapes]
    first[2] = first[2].bfloat16()

    def leaves():
        return [t.clone().requires_grad_() for t in first]
    ours, theirs = leaves(), leaves()

    def groups(p):
        return [{"params": p[:2], "weight_decay": 0.0}, {"params": p[2:], "lr": 2e-2}]
    opt = ssd.AdamW(groups(ours), lr=1e-2, state_bits=bits)
    ref = torch.optim.AdamW(groups(theirs), lr=1e-2)
    for t in range(3):
        for a, b in zip(ours, theirs):
            a.grad = torch.randn(a.shape, generator=g).cuda().to(a.dtype)
            b.grad = a.grad.clone()
        ours[3].grad = theirs[3].grad = None
        opt.step()
        ref.step()
    assert torch.equal(ours[3], first[3])
    for a, b in list(zip(ours, theirs))[:2] if bits == 32 else []:
        torch.testing.assert_close(a, b, rtol=1e-5, atol=1e-6)
    if bits == 8:  # 2^-4 of each average: the updates differ by an eighth of three steps of lr at most, p by rounding
        for a, b, lr in zip(ours[:2], theirs, (1e-2, 1e-2)):
            assert float((a - b).detach().abs().max()) <= 3 * lr * 0.25


@pytest.mark.parametrize("bits", [32, 8])
def test_optimiser_state_is_saved_and_loaded(bits):
    g = torch.Generator().manual_seed(2)
    p = torch.randn(40, 30, generator=g).cuda().bfloat16().requires_grad_()
    q = p.detach().clone().requires_grad_()
    a, b = ssd.AdamW([p], state_bits=bits), ssd.AdamW([q], state_bits=bits)

    def step(opt, t, seed):
        t.grad = torch.randn(40, 30, generator=torch.Generator().manual_seed(seed)).cuda().bfloat16()
        opt.step()
    step(a, p, 0)
    step(b, q, 0)
    fresh = ssd.AdamW([q], state_bits=bits)
    fresh.load_state_dict(b.state_dict())
    for seed in (1, 2):
        step(a, p, seed)
        step(fresh, q, seed)
    assert torch.equal(p, q)
    for k, v in a.state[p].items():
        w = fresh.state[q][k]
        assert v == w if k == "step" else (v.dtype == w.dtype and torch.equal(v.float(), w.float()))


def test_the_optimisers_step_is_not_captured():
    """A replay would repeat the step's number: refused, with nothing changed."""
    p = torch.ones(300, device="cuda", requires_grad=True)
    p.grad = torch.ones_like(p)
    opt = ssd.AdamW([p])
    opt.step()
    torch.cuda.synchronize()
    before, step = p.detach().clone(), opt.state[p]["step"]
    graph, other = torch.cuda.CUDAGraph(), torch.zeros(1, device="cuda")
    with torch.cuda.graph(graph):
        other += 1
        with pytest.raises(RuntimeError, match="step on the device"):
            opt.step()
    graph.replay()
    assert torch.equal(p, before) and opt.state[p]["step"] == step == 1 and float(other) == 1


def test_a_refused_step_is_not_counted():
    p = torch.ones(300, device="cuda", requires_grad=True)
    opt = ssd.AdamW([p])
    p.grad = torch.ones_like(p)
    opt.param_groups[0]["lr"] = -1.0
    with pytest.raises(ssd.SsdError):
        opt.step()
    assert opt.state[p]["step"] == 0 and torch.equal(p, torch.ones_like(p))
    opt.param_groups[0]["lr"] = 0.5
    opt.step()
    assert opt.state[p]["step"] == 1
