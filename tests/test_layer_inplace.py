"""Tensors that the layer operators overwrite are known to autograd as written:
a backward that had saved one raises instead of using the new values."""
import pytest
import torch

import state_space_sequence_cumsum_gb300 as ssd

pytestmark = pytest.mark.gpu


def rand(*shape):
    g = torch.Generator().manual_seed(len(shape))
    return torch.randn(shape, generator=g).cuda()


B, L, D, N = 2, 5, 8, 4


def conv_step(state):
    ssd.ssd_causal_conv_step(rand(B, D), rand(D, 4), state)


def scan_step(state):
    ssd.ssd_selective_scan_step(rand(B, D), rand(B, D), -rand(D, N).abs(), rand(B, N), rand(B, N), None, state)


def scan_in_place(state):
    ssd.ssd_selective_scan(rand(B, L, D), rand(B, L, D), -rand(D, N).abs(), rand(B, L, N), rand(B, L, N),
                           initial_state=state, final_state=state)


def scan_outputs(which):
    def call(t):
        ssd.ssd_selective_scan(rand(B, L, D), rand(B, L, D), -rand(D, N).abs(), rand(B, L, N), rand(B, L, N),
                               **{which: t})
    return call


CALLS = {  # name: (shape of what is written, call)
    "conv_step": ((B, 3, D), conv_step),
    "conv_step_out": ((B, 3, D), lambda t: ssd.ssd_causal_conv_step(rand(B, D), rand(D, 4), rand(B, 3, D), state_out=t)),
    "conv_step_y": ((B, D), lambda t: ssd.ssd_causal_conv_step(rand(B, D), rand(D, 4), rand(B, 3, D), y=t)),
    "conv_y": ((B, L, D), lambda t: ssd.ssd_causal_conv(rand(B, L, D), rand(D, 4), y=t)),
    "conv_final": ((B, 3, D), lambda t: ssd.ssd_causal_conv(rand(B, L, D), rand(D, 4), final_state=t)),
    "scan_step": ((B, D, N), scan_step),
    "scan_in_place": ((B, D, N), scan_in_place),
    "scan_y": ((B, L, D), scan_outputs("y")),
    "scan_chunk_states": ((B, 1, D, N), scan_outputs("chunk_states")),
    "norm_in_place": ((B, D), lambda t: ssd.ssd_block_norm(rand(B, D), t, rand(D), residual_out=t)),
    "norm_out": ((B, D), lambda t: ssd.ssd_block_norm(rand(B, D), rand(B, D), rand(D), out=t)),
}


@pytest.mark.parametrize("name", CALLS)
def test_a_saved_tensor_that_is_overwritten_raises(name):
    shape, call = CALLS[name]
    t, w = rand(*shape), rand(*shape).requires_grad_(True)
    before = t._version
    loss = (t * w).sum()  # saves t
    call(t)
    assert t._version > before
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_what_is_not_given_is_not_marked():
    x, w, init = rand(B, L, D), rand(D, 4), rand(B, 3, D)
    versions = [t._version for t in (x, w, init)]
    ssd.ssd_causal_conv(x, w, initial_state=init, return_final_state=True)
    ssd.ssd_causal_conv_step(x[:, 0], w, init, state_out=torch.empty_like(init))
    assert [t._version for t in (x, w, init)] == versions


def test_a_refused_call_marks_nothing():
    y, x = rand(B, L, D), rand(B, L, D)
    before = y._version
    with pytest.raises(ssd.SsdError):
        ssd.ssd_causal_conv(x, rand(D, 5), y=y)
    with pytest.raises(ssd.SsdError):
        ssd.ssd_causal_conv(x, rand(D, 4), y=x)
    assert y._version == before and x._version == 0


def test_inference_tensors_are_updated_in_and_out_of_inference_mode():
    with torch.inference_mode():
        state = torch.zeros(B, 3, D, device="cuda")
        ssd.ssd_causal_conv_step(rand(B, D), rand(D, 4), state)
    assert torch.equal(state[:, 2], rand(B, D))
    ssd.ssd_causal_conv_step(rand(B, D), rand(D, 4), state)
    assert torch.equal(state[:, 1:], torch.stack([rand(B, D)] * 2, 1))
