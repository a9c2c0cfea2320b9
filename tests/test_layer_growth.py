"""States that grow: a positive rate (or step times rate) is a recurrence like
any other, and a state that is still zero stays zero however much a run of
tokens would grow it.  Every number of these cases is finite in f32.

The factors are up to e^2 a token over at most 20 tokens from the first input,
each with a rounding of the exponent (40 x 2^-24 relative) and the exponential's
2^-22: 20 (40 x 2^-24 + 2^-22) < 5.3e-5 of the result's scale, under the
tolerances of the scan's other tests, which are used here."""
import pytest
import torch

from oracle import layer
import state_space_sequence_cumsum_gb300 as ssd
from test_layer import SCAN, close

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sign", ["rate", "step"])
@pytest.mark.parametrize("L,D,N", [(2048, 8, 4), (1500, 20, 16)])
def test_growth_across_segments(L, D, N, sign):
    """Inputs in the last 20 tokens and output gradients in the first 20; in
    between, segments whose whole factor is beyond f32."""
    g = torch.Generator().manual_seed(L)
    A = torch.rand(D, N, generator=g) + 1.0
    dt = torch.ones(1, L, D)
    if sign == "step":
        A, dt = -A, -dt
    u, dy = torch.zeros(1, L, D), torch.zeros(1, L, D)
    u[:, -20:] = torch.randn(1, 20, D, generator=g)
    dy[:, :20] = torch.randn(1, 20, D, generator=g)
    B, C = (torch.randn(1, L, 1, N, generator=g) for _ in range(2))
    args = [t.cuda() for t in (u, dt, A, B, C)]
    y, fin, kept = ssd.ssd_selective_scan(*args, dt_softplus=False, return_chunk_states=True)
    wy, h = layer.scan(u, dt, A, B, C, softplus=False)
    close(y, wy, SCAN)
    close(fin, h[:, -1], SCAN)
    want = layer.scan_bwd(u, dt, A, B, C, dy, softplus=False)
    for states in (kept, None):
        got = ssd.ssd_selective_scan_bwd(*args, None, dy.cuda(), dt_softplus=False, chunk_states=states)
        for k, v in got.items():
            if v is not None:
                close(v, want[k], 2 * SCAN)
