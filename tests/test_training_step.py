"""The 8-bit projections, the operators between them and the optimiser's step in a
row, as a training step uses them, against the float64 definitions in a row.

Tolerances.  In f32 each operator is within some 2^-20 of its definition, so a
value that is rounded to 8 bits may fall to the other side of a border, a step of
2^-3 of itself at most, in one of some 10^6 cases for each such rounding: the
norm of a result is off by far less than 2^-3 sqrt(10^-5) = 4e-4 of itself."""
import importlib.util
import math
import os

import numpy as np
import pytest
import torch

import state_space_sequence_cumsum_gb300 as ssd
from oracle import blocks, layer

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NEAR = 4e-4


def near(got, want):
    got = got.detach().double().cpu().numpy()
    assert got.shape == want.shape
    assert np.linalg.norm(got - want) <= NEAR * np.linalg.norm(want), np.linalg.norm(got - want) / np.linalg.norm(want)


@pytest.mark.parametrize("b,L,dim,inner", [(2, 150, 200, 333), (1, 1, 64, 130), (3, 700, 129, 256)])
def test_two_projections_a_convolution_and_the_step(b, L, dim, inner):
    g = torch.Generator().manual_seed(0)

    def r(*shape, scale=1.0):
        return (torch.randn(shape, generator=g) * scale).cuda()
    x, dy = r(b, L, dim), r(b, L, dim)
    params = [r(inner, dim, scale=dim ** -0.5), r(inner, 4, scale=0.5), r(inner), r(dim, inner, scale=inner ** -0.5)]
    w_in, conv, bias, w_out = (p.requires_grad_() for p in params)
    x.requires_grad_()
    u = ssd.ProjectionFunction.apply(x, w_in)
    c, _ = ssd.CausalConvFunction.apply(u, conv, bias)
    y = ssd.ProjectionFunction.apply(c, w_out)
    y.backward(dy)

    f = {k: v.detach().double().cpu().numpy() for k, v in dict(x=x, dy=dy, w_in=w_in, conv=conv, bias=bias, w_out=w_out).items()}
    flat = f["x"].reshape(-1, dim)
    vin, vout = (blocks.values(*blocks.quantise(f[k], tile=True)) for k in ("w_in", "w_out"))
    fu = blocks.projection(flat, vin).reshape(b, L, inner)
    fc, _ = layer.conv(fu, f["conv"], f["bias"])
    fy = blocks.projection(fc.reshape(-1, inner), vout)
    near(y, fy.reshape(b, L, dim))
    dc, dout = blocks.projection_bwd(fc.reshape(-1, inner), vout, f["dy"].reshape(-1, dim))
    grads = layer.conv_bwd(fu, f["conv"], dc.reshape(b, L, inner), f["bias"])
    du, dconv, dbias = grads["dx"], grads["dweight"], grads["dbias"]
    dx, din = blocks.projection_bwd(flat, vin, du.reshape(-1, inner))
    near(x.grad, dx.reshape(b, L, dim))
    for p, want in ((w_in, din), (conv, dconv), (bias, dbias), (w_out, dout)):
        near(p.grad, want)

    # the optimiser's step from these gradients, for both kinds of states
    for bits in (32, 8):
        again = [p.detach().clone().requires_grad_() for p in params]
        for a, p in zip(again, params):
            a.grad = p.grad.clone()
        opt = ssd.AdamW(again, lr=1e-2, weight_decay=0.1, state_bits=bits)
        opt.step()
        for a, p in zip(again, params):
            p0, gr = (t.detach().double().cpu().numpy() for t in (p, p.grad))
            zero = np.zeros_like(p0)
            want, _, _ = blocks.adamw(p0, gr, zero, zero, 1, 1e-2, (0.9, 0.999), 1e-8, 0.1)
            assert np.abs(a.detach().double().cpu().numpy() - want).max() <= 2.0 ** -18 * (1e-2 + np.abs(p0).max())


def test_example_in_8_bits():
    """The example model with 8-bit projections: it runs, its gradients are the
    plain model's up to the roundings to 8 bits, and it generates."""
    spec = importlib.util.spec_from_file_location("selective_model", os.path.join(ROOT, "examples", "selective_model.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    grads = []
    for eight_bit in (False, True):
        torch.manual_seed(0)
        model = m.Model(eight_bit=eight_bit).cuda()
        data = torch.randint(0, 64, (4, 65), generator=torch.Generator().manual_seed(1)).cuda()
        logits, _ = model(data[:, :-1])
        torch.nn.functional.cross_entropy(logits.reshape(-1, 64), data[:, 1:].reshape(-1)).backward()
        grads.append([p.grad.double() for p in model.parameters()])
    for a, b in zip(*grads):
        assert torch.isfinite(b).all()
        # rounding errors of 2^-4 a value at most, 2^-5.8 in the mean square, in a dozen
        # roundings between a parameter and the loss
        assert float((a - b).norm()) <= 12 ** 0.5 * 2.0 ** -4 * float(a.norm())
    losses, gap, right = m.main(steps=3, seqlen=32, sequences=4, generate=4, quiet=True, eight_bit=True)
    assert len(losses) == 3 and all(math.isfinite(v) for v in losses) and math.isfinite(gap)
