"""The float64 definitions of the 8-bit projections and of the optimiser's step:
hand-worked values, the types' own grids, and identities."""
import numpy as np
import pytest
import torch

from oracle import blocks


@pytest.mark.parametrize("kind,dtype", [(blocks.E4M3, torch.float8_e4m3fn), (blocks.E5M2, torch.float8_e5m2)])
def test_rounding_is_the_type_s(kind, dtype):
    """Every value of the type is kept, and a point between two neighbours goes
    to the nearer one, the middle to the even code."""
    codes = torch.arange(0, 127 if dtype == torch.float8_e4m3fn else 124, dtype=torch.uint8)
    grid = codes.view(dtype).double().numpy()
    assert np.array_equal(blocks.round8(grid, kind), grid) and grid[-1] == kind[0]
    mid = (grid[1:] + grid[:-1]) / 2
    even = np.where(np.arange(len(mid)) % 2 == 0, grid[:-1], grid[1:])
    assert np.array_equal(blocks.round8(mid, kind), even)
    assert np.array_equal(blocks.round8(mid * (1 + 1e-12), kind), grid[1:])
    assert np.array_equal(blocks.round8(-mid * (1 - 1e-12), kind), -grid[:-1])


@pytest.mark.parametrize("amax,scale", [(448.0, 1.0), (448.1, 2.0), (224.0, 0.5), (0.0, 2.0 ** -118), (1.0, 2.0 ** -8),
                                        (1.75, 2.0 ** -8), (1.76, 2.0 ** -7), (2.0 ** -130, 2.0 ** -118)])
def test_scale_is_the_least_power_of_two(amax, scale):
    assert blocks.block_scale(amax) == scale


def test_blocks_and_transposes():
    rng = np.random.default_rng(0)
    x = rng.normal(size=(200, 300)) * np.exp(rng.normal(size=(200, 1)) * 3)
    q, s = blocks.quantise(x)
    assert s.shape == (200, 3) and (np.abs(blocks.values(q, s) - x) <= np.abs(x).max() * 2.0 ** -4).all()
    # relative 2^-4 for normal values
    normal = np.abs(q) >= 2.0 ** -6
    assert (np.abs(blocks.values(q, s) - x)[normal] <= 2.0 ** -4 * np.abs(x)[normal]).all()
    q, s = blocks.quantise(x, tile=True)
    qt, st = blocks.quantise(x.T, tile=True)
    assert s.shape == (2, 3) and np.array_equal(q.T, qt) and np.array_equal(s.T, st)
    x[7, 130] = np.inf
    q, s = blocks.quantise(x)
    assert np.isnan(s[7, 1]) and np.isnan(q[7, 128:256]).all() and np.isfinite(np.delete(q, 7, 0)).all()
    assert np.isfinite(q[7, :128]).all()


def test_projection_gradients_are_those_of_its_products():
    """With values that 8 bits hold exactly, quantising changes nothing, and the
    gradients are those of a plain product by central differences."""
    rng = np.random.default_rng(1)
    x, w, dy = (rng.integers(-8, 9, size=s).astype(float) for s in ((5, 7), (3, 7), (5, 3)))
    assert np.array_equal(blocks.projection(x, w), x @ w.T)
    dx, dw = blocks.projection_bwd(x, w, dy)
    h = 1e-3
    for t, d in ((x, dx), (w, dw)):
        for i in np.ndindex(*t.shape):
            t[i] += h
            up = (x @ w.T * dy).sum()
            t[i] -= 2 * h
            down = (x @ w.T * dy).sum()
            t[i] += h
            assert abs((up - down) / (2 * h) - d[i]) < 1e-8


def test_states_in_8_bits():
    x = np.array([448.0, 1.0, 2.0 ** -12, 0.0, -3.0])
    q, s = blocks.quantise_state(x)
    assert s.tolist() == [1.0] and q.tolist() == [448.0, 1.0, 0.0, 0.0, -3.0]
    q, s = blocks.quantise_state(np.abs(x), root=True)
    assert q.tolist() == [448.0, 1.0, 2.0 ** -9, 0.0, 3.0]
    q, s = blocks.quantise_state(np.full(300, 2.0 ** -101))
    assert not q.any() and s.tolist() == [0.0, 0.0]


def test_adamw_is_torch_s():
    """Three steps against torch's optimiser in float64."""
    rng = np.random.default_rng(2)
    p0 = rng.normal(size=40)
    p = torch.tensor(p0, requires_grad=True)
    kw = dict(lr=1e-2, betas=(0.8, 0.9), eps=1e-6, weight_decay=0.3)
    opt = torch.optim.AdamW([p], foreach=False, **kw)
    q, m, v = p0, np.zeros(40), np.zeros(40)
    for t in range(1, 4):
        g = rng.normal(size=40)
        p.grad = torch.tensor(g * 0.5)
        opt.step()
        q, m, v = blocks.adamw(q, g, m, v, t, grad_scale=0.5, **kw)
        assert np.abs(q - p.detach().numpy()).max() < 1e-14
