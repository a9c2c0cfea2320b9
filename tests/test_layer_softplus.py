"""The scan's step through softplus, against 64 bits over the range of steps.

A state that starts at zero takes delta u B, so with u = B = 1 it is delta
itself.  e^-|x| is formed as 2^t, t = -|x| log2(e): the constant's and the
product's roundings are |x| 2^-24 each of the exponential, 2^t is off by 2^-22
and what follows (a reciprocal and five roundings) by 2^-21 at most, all
relative; the polynomial's 1e-8 is far below.  Past -87 the result leaves the
normal numbers and only has to vanish."""
import pytest
import torch

import state_space_sequence_cumsum_gb300 as ssd

pytestmark = pytest.mark.gpu


def delta_of(x, form):
    n, dev = x.numel(), "cuda"
    one, A = torch.ones(1, 1, n, device=dev), -torch.ones(n, 1, device=dev)
    m = torch.ones(1, 1, 1, device=dev)
    dt = x.reshape(1, 1, n).cuda()
    if form == "prompt":
        return ssd.ssd_selective_scan(one, dt, A, m, m)[1].reshape(-1)
    state = torch.zeros(1, n, 1, device=dev)
    return ssd.ssd_selective_scan_step(one[:, 0], dt[:, 0], A, m[:, 0], m[:, 0], None, state)[1].reshape(-1)


@pytest.mark.parametrize("form", ["prompt", "token"])
def test_relative_error_over_the_range(form):
    x = torch.linspace(-80, 80, 100001)
    got = delta_of(x, form).cpu().double()
    x = x.double()
    want = torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))
    err = (got - want).abs() / want
    bound = x.abs() * 2.0 ** -23 + 2.0 ** -22 + 2.0 ** -21
    assert bool((err <= bound).all())


def test_ends_of_the_range():
    got = delta_of(torch.tensor([-float("inf"), -1e4, -120.0, 0.0, 1e4, 3e38, float("inf")]), "prompt").cpu()
    assert float(got[:3].abs().max()) < 1e-37 and got[4:].tolist() == [1e4, float(torch.tensor(3e38)), float("inf")]
    assert abs(float(got[3]) - 0.6931471805599453) < 1e-6
