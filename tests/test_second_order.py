"""Gradients of gradients: the operators' backward passes are kernels, which
autograd cannot differentiate.  A derivative through one raises, first-order
results (create_graph or not) are the same, and nothing is dropped silently."""
import pytest
import torch

import state_space_sequence_cumsum_gb300 as ssd
from state_space_sequence_cumsum_gb300._autograd import first_order


class Cube(torch.autograd.Function):
    """x^3 y with a backward of constants, as a kernel's is."""

    @staticmethod
    def forward(ctx, x, y, power):
        ctx.save_for_backward(x, y)
        return x ** 3 * y

    @staticmethod
    @first_order
    def backward(ctx, g):
        x, y = ctx.saved_tensors
        return 3 * g * x * x * y, g * x ** 3, None


def test_a_marked_backward_refuses_to_be_differentiated():
    x, y = torch.tensor([2.0, -1.0], requires_grad=True), torch.tensor([3.0, 0.5])
    out = Cube.apply(x, y, None)
    (once,) = torch.autograd.grad(out.sum(), x, retain_graph=True)
    assert not once.requires_grad and once.tolist() == [36.0, 1.5]
    (kept,) = torch.autograd.grad(out.sum(), x, create_graph=True)
    assert torch.equal(kept, once)
    with pytest.raises(RuntimeError, match="Cube has no second-order"):
        (kept.square().sum() + x.sum()).backward()


def cases():
    g = torch.Generator().manual_seed(0)

    def r(*shape):
        return torch.randn(shape, generator=g).cuda()
    B, L, D, N = 2, 20, 8, 4
    return {
        "CausalConvFunction": (r(B, L, D), r(D, 4), r(D), None),
        "SelectiveScanFunction": (r(B, L, D), r(B, L, D), -r(D, N).abs(), r(B, L, N), r(B, L, N), r(D), r(B, L, D)),
        "BlockNormFunction": (r(B * L, D), r(B * L, D), r(D), r(D)),
        "SsdFunction": (r(B, L, 2, D), r(B, L, 2).abs() * 0.1, -r(2).abs(), r(B, L, 1, N), r(B, L, 1, N), r(2)),
    }


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["CausalConvFunction", "SelectiveScanFunction", "BlockNormFunction", "SsdFunction"])
def test_gradient_penalty_raises(name):
    args = cases()[name]
    x = args[0].requires_grad_(True)

    def loss():
        return getattr(ssd, name).apply(*args)[0].sum()
    (once,) = torch.autograd.grad(loss(), x)
    (kept,) = torch.autograd.grad(loss(), x, create_graph=True)
    assert torch.equal(kept, once)
    with pytest.raises(RuntimeError, match=f"{name} has no second-order"):
        (loss() + kept.square().sum()).backward()
