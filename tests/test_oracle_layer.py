"""The float64 references of the layer operators: hand-worked values and every
gradient against central differences (CPU only).

Central differences with step 1e-5 of smooth functions in float64: the
truncation error is about 1e-10 and the rounding error about 1e-16 / 1e-5
times the loss, so 1e-6 relative to the largest gradient entry is ample."""
import numpy as np
import pytest

from oracle import layer


def differences(f, a, step=1e-5):
    g = np.zeros_like(a)
    for i in np.ndindex(a.shape):
        keep = a[i]
        a[i] = keep + step
        up = f()
        a[i] = keep - step
        g[i] = (up - f()) / (2 * step)
        a[i] = keep
    return g


def agree(got, want):
    assert got.shape == want.shape
    assert np.max(np.abs(got - want)) <= 1e-6 * max(1.0, np.max(np.abs(want)))


def test_conv_by_hand():
    y, fin = layer.conv([[[1.0], [2.0], [3.0]]], [[10.0, 1.0]], [0.5], [[[4.0]]], silu=False)
    assert y.reshape(-1).tolist() == [41.5, 12.5, 23.5] and fin.reshape(-1).tolist() == [3.0]


def test_scan_by_hand():
    # one channel, one state, delta = 1 without softplus, exp(A) = 1/2
    A = [[np.log(0.5)]]
    one = np.ones((1, 3, 1))
    y, h = layer.scan(2 * one, one, A, one[..., None], 3 * one[..., None], [1.0], softplus=False)
    assert np.allclose(h.reshape(-1), [0, 2, 3, 3.5]) and np.allclose(y.reshape(-1), [8, 11, 12.5])


@pytest.mark.parametrize("W,L,silu,carry", [(2, 3, True, True), (3, 1, False, True), (4, 2, True, True),
                                            (4, 6, True, False)])
def test_conv_gradient(W, L, silu, carry):
    r = np.random.default_rng(W * 10 + L)
    x, w, b = r.normal(size=(2, L, 3)), r.normal(size=(3, W)), r.normal(size=3)
    init = r.normal(size=(2, W - 1, 3)) if carry else None
    dy, df = r.normal(size=(2, L, 3)), r.normal(size=(2, W - 1, 3))

    def loss():
        y, fin = layer.conv(x, w, b, init, silu)
        return (y * dy).sum() + (fin * df).sum()

    g = layer.conv_bwd(x, w, dy, b, init, df, silu)
    for name, a in (("dx", x), ("dweight", w), ("dbias", b)) + ((("dinit", init),) if carry else ()):
        agree(g[name], differences(loss, a))


@pytest.mark.parametrize("L,N,G,gated,softplus,skip", [(5, 3, 1, True, True, True), (1, 2, 2, False, True, False),
                                                       (4, 1, 2, True, False, True)])
def test_scan_gradient(L, N, G, gated, softplus, skip):
    r = np.random.default_rng(L)
    dim = 4
    u, dt, z = (r.normal(size=(2, L, dim)) for _ in range(3))
    A, init, df = -np.exp(r.normal(size=(dim, N))), r.normal(size=(2, dim, N)), r.normal(size=(2, dim, N))
    Bm, Cm = r.normal(size=(2, L, G, N)), r.normal(size=(2, L, G, N))
    D, bias, dy = r.normal(size=dim), r.normal(size=dim), r.normal(size=(2, L, dim))
    D, z = (D if skip else None), (z if gated else None)

    def loss():
        y, h = layer.scan(u, dt, A, Bm, Cm, D, z, bias, softplus, init)
        return (y * dy).sum() + (h[:, -1] * df).sum()

    g = layer.scan_bwd(u, dt, A, Bm, Cm, dy, D, z, bias, softplus, init, df)
    pairs = {"du": u, "ddt": dt, "dA": A, "dB": Bm, "dC": Cm, "ddt_bias": bias, "dinit": init}
    if skip:
        pairs["dD"] = D
    if gated:
        pairs["dz"] = z
    for name, a in pairs.items():
        agree(g[name], differences(loss, a))


@pytest.mark.parametrize("post,rows", [(True, 2), (True, 6), (False, 1), (True, 0), (False, 0)])
def test_block_norm_gradient(post, rows):
    r = np.random.default_rng(rows)
    y, res, dout, dr = (r.normal(size=(6, 5)) for _ in range(4))
    w, pw = r.normal(size=5), (r.normal(size=5) if post else None)
    gate = r.normal(size=(rows, 5)) if rows else None

    def loss():
        out, rr = layer.block_norm(y, res, w, pw, gate, 0.3, 1e-3)
        return (out * dout).sum() + (rr * dr).sum()

    _, rr = layer.block_norm(y, res, w, pw, gate, 0.3, 1e-3)
    g = layer.block_norm_bwd(y, rr, w, dout, dr, pw, gate, 0.3, 1e-3)
    pairs = {"dy": y, "dresidual": res, "dweight": w}
    if post:
        pairs["dpost_weight"] = pw
    if rows:
        pairs["dgate"] = gate
    for name, a in pairs.items():
        agree(g[name], differences(loss, a))
