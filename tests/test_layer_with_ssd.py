"""A Mamba-2 layer's convolution and its scan in a row: one convolution over
the channels of x, B and C, then ssd_fwd (which takes them contiguous, so each
slice is copied), trained through both and continued token by token.

Tolerances.  The scan's f32 results and gradients are held to 1e-4 of their rms
by their own tests.  Through the convolution's backward such an error of dy
reaches dx multiplied by at most sum |w| max |silu'| < 2.2, against an rms of dx
that is at least half of dy's here; with the same again for the convolution's
own error in the scan's inputs, 1e-3 of (element + rms) bounds every gradient,
and 3e-4 every output."""
import numpy as np
import pytest
import torch

import oracle
from oracle import layer
import state_space_sequence_cumsum_gb300 as ssd

pytestmark = pytest.mark.gpu


def near(got, want, tol):
    g = got.detach().to("cpu", torch.float64).numpy()
    assert g.shape == want.shape and np.all(np.isfinite(g))
    assert np.max(np.abs(g - want) - tol * (np.abs(want) + np.sqrt(np.mean(want * want)))) <= 0.0


def parts(t, H, P, G, S):
    """[..., H P + 2 G S] -> x [..., H, P], B and C [..., G, S]."""
    x, B, C = t.split((H * P, G * S, G * S), -1)
    return x.unflatten(-1, (H, P)), B.unflatten(-1, (G, S)), C.unflatten(-1, (G, S))


@pytest.mark.parametrize("B,L,H,P,G,S", [(2, 150, 4, 16, 2, 32), (1, 70, 3, 8, 1, 16), (1, 1, 2, 8, 1, 16)])
def test_convolution_then_scan(B, L, H, P, G, S):
    g = torch.Generator().manual_seed(L)

    def r(*shape, std=1.0):
        return torch.randn(shape, generator=g) * std
    dim = H * P + 2 * G * S
    v, w, bias, carry = r(B, L + 1, dim), r(dim, 4, std=0.5), r(dim, std=0.3), r(B, 3, dim)
    dt, A, D, init = r(B, L + 1, H).abs() * 0.1, -r(H).abs() - 0.1, r(H), r(B, H, P, S, std=0.3)
    dy, dh = r(B, L, H, P), r(B, H, P, S)
    # in 64 bits
    u, _ = layer.conv(v, w, bias, carry)
    x, Bm, Cm = parts(torch.from_numpy(u), H, P, G, S)
    now = [t[:, :L].contiguous() for t in (x, Bm, Cm)]
    ref = oracle.fwd(now[0], dt[:, :L].contiguous(), A, now[1], now[2], D, 64, init=init)
    gr = oracle.bwd(now[0], dt[:, :L].contiguous(), A, now[1], now[2], D, dy, init=init, dfinal=dh)
    du = np.concatenate([gr[k].reshape(B, L, -1) for k in ("dx", "dB", "dC")], -1)
    gc = layer.conv_bwd(v[:, :L], w, du, bias, carry)
    # trained through both
    leaves = [t.cuda().requires_grad_(True) for t in (v[:, :L].contiguous(), w, bias, carry, dt[:, :L].contiguous(), A, D,
                                                     init)]
    vd, wd, bd, cd, dtd, Ad, Dd, hd = leaves
    ud, state = ssd.CausalConvFunction.apply(vd, wd, bd, cd)
    xd, Bd, Cd = (t.contiguous() for t in parts(ud, H, P, G, S))
    y, final = ssd.SsdFunction.apply(xd, dtd, Ad, Bd, Cd, Dd, hd)
    near(y, ref["y"], 3e-4)
    near(final, ref["final_state"], 3e-4)
    torch.autograd.backward([y, final], [dy.cuda(), dh.cuda()])
    for t, want in zip(leaves, (gc["dx"], gc["dweight"], gc["dbias"], gc["dinit"], gr["ddt"], gr["dA"], gr["dD"],
                                gr["dinit"])):
        near(t.grad, want, 1e-3)
    # one more token through both single-token forms
    with torch.no_grad():
        one, _ = ssd.ssd_causal_conv_step(v[:, L].cuda(), wd.detach(), state, bd.detach())
        near(one, u[:, L], 3e-4)
        x1, B1, C1 = (t.contiguous() for t in parts(one, H, P, G, S))
        y1, final = ssd.ssd_decode_step(x1, dt[:, L].contiguous().cuda(), A.cuda(), B1, C1, D.cuda(), final.detach())
    ref = oracle.fwd(x.contiguous(), dt, A, Bm.contiguous(), Cm.contiguous(), D, 64, init=init)
    near(y1, ref["y"][:, L], 3e-4)
    near(final, ref["final_state"], 3e-4)
    assert ssd.ssd_stream_status() == 0
