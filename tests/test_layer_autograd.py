"""What the autograd functions ask of the kernels: no chunk states without a
gradient to come, no gradient of a state that needs none, no zeros read for an
output that was not used."""
import pytest
import torch

import state_space_sequence_cumsum_gb300 as ssd
from state_space_sequence_cumsum_gb300 import layer

B, L, D, N = 2, 40, 8, 4


class Recorded(Exception):
    pass


@pytest.fixture
def scan_calls(monkeypatch):
    """ssd_selective_scan's requests for chunk states, without its kernels."""
    calls = []

    def fake(*args, return_chunk_states=False, **kw):
        calls.append(return_chunk_states)
        u = args[0]
        return torch.zeros_like(u), torch.zeros(B, D, N), torch.zeros(1) if return_chunk_states else None
    monkeypatch.setattr(layer, "ssd_selective_scan", fake)
    return calls


def scan_args(grad=False):
    t = [torch.randn(s) for s in ((B, L, D), (B, L, D), (D, N), (B, L, N), (B, L, N))]
    t[2].requires_grad_(grad)
    return t


def test_chunk_states_are_kept_for_a_backward_only(scan_calls):
    apply = ssd.SelectiveScanFunction.apply
    with torch.no_grad():
        y, final = apply(*scan_args(True))
    apply(*scan_args(False))
    assert scan_calls == [False, False] and y.shape == (B, L, D) and final.shape == (B, D, N)
    y, final = apply(*scan_args(True), None, None, None, None, False)
    assert scan_calls == [False, False, True] and y.requires_grad and final.requires_grad


@pytest.mark.parametrize("name", ["ssd_causal_conv", "ssd_selective_scan"])
@pytest.mark.parametrize("wanted", [True, False])
def test_unused_final_state_and_unwanted_state_gradient(monkeypatch, name, wanted):
    """The backward is given None for the final state's gradient and asked for
    the initial state's only where that needs one."""
    seen = {}

    def forward(*args, **kw):
        u = args[0]
        final = torch.zeros(B, 3, D) if "conv" in name else torch.zeros(B, D, N)
        return (torch.zeros_like(u), final) + ((torch.zeros(1),) if "scan" in name else ())

    def backward(*args, want_dinit, **kw):
        seen.update(args=args, want=want_dinit)
        raise Recorded
    monkeypatch.setattr(layer, name, forward)
    monkeypatch.setattr(layer, name + "_bwd", backward)
    if "conv" in name:
        init = torch.zeros(B, 3, D, requires_grad=wanted)
        x = torch.randn(B, L, D, requires_grad=True)
        y, final = ssd.CausalConvFunction.apply(x, torch.randn(D, 4), None, init)
        at_dy, at_dfinal = 2, 6
    else:
        init = torch.zeros(B, D, N, requires_grad=wanted)
        y, final = ssd.SelectiveScanFunction.apply(*scan_args(True), None, None, None, init)
        at_dy, at_dfinal = 6, 11
    with pytest.raises(Recorded):
        y.sum().backward(retain_graph=True)
    assert seen["want"] is wanted and seen["args"][at_dfinal] is None and bool((seen["args"][at_dy] == 1).all())
    with pytest.raises(Recorded):
        final.sum().backward()
    assert bool((seen["args"][at_dfinal] == 1).all()) and bool((seen["args"][at_dy] == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("use", ["first", "second"])
@pytest.mark.parametrize("name", ["conv", "scan", "norm"])
def test_gradients_of_one_output_alone(name, use):
    """The same as with an explicit zero gradient for the other output."""
    g = torch.Generator().manual_seed(1)

    def r(*shape, neg=False):
        t = torch.randn(shape, generator=g)
        return (-t.abs() if neg else t).cuda().requires_grad_(True)
    args, f = {
        "conv": lambda: ((r(B, L, D), r(D, 4), r(D), r(B, 3, D)), ssd.CausalConvFunction),
        "scan": lambda: ((r(B, L, D), r(B, L, D), r(D, N, neg=True), r(B, L, N), r(B, L, N), r(D), r(B, L, D), r(D),
                          r(B, D, N)), ssd.SelectiveScanFunction),
        "norm": lambda: ((r(B * L, D), r(B * L, D), r(D), r(D), r(B, D)), ssd.BlockNormFunction),
    }[name]()
    first, second = f.apply(*args)
    used = first if use == "first" else second
    got = torch.autograd.grad(used.square().sum(), args, allow_unused=True)
    first, second = f.apply(*args)
    used, other = (first, second) if use == "first" else (second, first)
    want = torch.autograd.grad(used.square().sum() + 0.0 * other.sum(), args)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
