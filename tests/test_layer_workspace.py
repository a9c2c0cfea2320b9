"""A Workspace object used on more than one stream: the buffer that it grows out
of stays with the stream that still works in it."""
import pytest
import torch

import state_space_sequence_cumsum_gb300 as ssd

pytestmark = pytest.mark.gpu


def calls():
    g = torch.Generator(device="cuda").manual_seed(0)

    def r(*shape):
        return torch.randn(shape, generator=g, device="cuda")
    x, dy, w = r(2, 300, 96), r(2, 300, 96), r(96, 4)
    dt, z, A, B, C = r(2, 300, 96), r(2, 300, 96), -r(96, 16).abs(), r(2, 300, 16), r(2, 300, 16)
    y, gate = r(600, 96), r(2, 96)
    return {
        "conv": lambda **k: ssd.ssd_causal_conv_bwd(x, w, dy, **k),
        "scan": lambda **k: ssd.ssd_selective_scan_bwd(x, dt, A, B, C, None, dy, z, **k),
        "norm": lambda **k: ssd.ssd_block_norm_bwd(y, y, w[:, 0].contiguous(), dy.reshape(600, 96), gate=gate, **k),
    }


@pytest.mark.parametrize("name", ["conv", "scan", "norm"])
def test_workspace_outgrown_while_another_stream_uses_it(name):
    call = calls()[name]
    want = call()
    ws = ssd.Workspace()
    call(workspace=ws)                        # allocated from the current stream's pool
    old, size = ws.buf.data_ptr(), ws.buf.numel()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)        # about 0.2 s, so that the call below waits
    got = call(workspace=ws, stream=side)
    ws.get(4 * size, ws.buf.device)           # grown: the buffer goes back to the allocator
    assert not side.query()
    # enough of its size to take every free block of the pool that fits
    others = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(64)]
    assert not any(t.data_ptr() < old + size and old < t.data_ptr() + size for t in others)
    for t in others:
        t.fill_(255)
    side.synchronize()
    for k in want:
        if want[k] is not None:
            assert torch.equal(got[k], want[k])


def test_one_workspace_on_two_streams_in_order():
    ws, side = ssd.Workspace(), torch.cuda.Stream()
    for name, call in calls().items():
        want = call()
        side.wait_stream(torch.cuda.current_stream())
        a = call(workspace=ws, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        b = call(workspace=ws)
        for k in want:
            if want[k] is not None:
                assert torch.equal(a[k], want[k]) and torch.equal(b[k], want[k])
