"""The 8-bit projections on the GPU against the float64 definitions.

Tolerances.  Quantising rounds each value once and its scale is a power of two,
so values and scales are the definition's, bit for bit.  A product of two 8-bit
values is exact in f32; a block's 128 products are summed in the tensor core and
at most ceil(k / 128) blocks in f32, each times two scales: an element is off by
at most (128 + ceil(k / 128) + 3) 2^-24 of the sum of its terms' magnitudes,
and by half a step (2^-8 for bf16) of its own value."""
import math

import numpy as np
import pytest
import torch

import state_space_sequence_cumsum_gb300 as ssd
from oracle import blocks

pytestmark = pytest.mark.gpu

BF, F32, E4, E5 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.float8_e5m2
KINDS = {E4: blocks.E4M3, E5: blocks.E5M2}
HALF_STEP = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def np64(t):
    return t.detach().float().double().cpu().numpy()


def tokens(rows, cols, dtype=BF, seed=0, row=None):
    """Channels and tokens of different sizes; `row` elements between rows."""
    g = torch.Generator().manual_seed(seed)
    t = torch.randn(rows, cols, generator=g) * torch.exp(torch.randn(cols, generator=g)) * \
        torch.exp(2 * torch.randn(rows, 1, generator=g))
    t = t.to(dtype).cuda()
    if row is None:
        return t
    wide = torch.full((rows, row), 7.0, dtype=dtype, device="cuda")
    wide[:, row - cols:] = t
    return wide[:, row - cols:]


def check(got, want, magnitude, k):
    """magnitude: the sum of the terms' magnitudes of each element."""
    bound = (128 + -(-k // 128) + 3) * 2.0 ** -24 * magnitude + HALF_STEP[got.dtype] * np.abs(want) * (1 + 2.0 ** -12)
    got = np64(got)
    assert got.shape == want.shape and np.isfinite(got).all()
    assert (np.abs(got - want) <= bound).all(), np.max(np.abs(got - want) / np.maximum(bound, 1e-300))
    assert ssd.ssd_stream_status() == 0


def check_product(got, a, b):
    check(got, a @ b.T, np.abs(a) @ np.abs(b).T, a.shape[1])


# --------------------------------------------------------------- quantising

def check_quantised(x, tile, fp8=E4):
    q, s, qt, st = ssd.ssd_block_quantize(x, tile=tile, fp8=fp8, want_t=True)
    for got_q, got_s, like in ((q, s, x), (qt, st, x.t())):
        want_q, want_s = blocks.quantise(np64(like), tile, KINDS[fp8])
        assert got_q.dtype == fp8 and got_s.dtype == F32
        np.testing.assert_array_equal(np64(got_q), want_q)
        np.testing.assert_array_equal(np64(got_s), want_s)


@pytest.mark.parametrize("rows,cols,row", [(1, 1, None), (1, 300, None), (128, 128, None), (129, 127, 131), (37, 260, 264),
                                           (300, 129, None), (257, 1000, 1001), (16, 16, 20), (500, 4, None)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("tile", [False, True])
def test_quantise(rows, cols, row, dtype, tile):
    check_quantised(tokens(rows, cols, dtype, row=row), tile)


@pytest.mark.parametrize("tile", [False, True])
def test_quantise_e5m2(tile):
    check_quantised(tokens(200, 333, F32), tile, E5)


@pytest.mark.parametrize("fp8", [E4, E5])
@pytest.mark.parametrize("tile", [False, True])
def test_quantise_borders(tile, fp8):
    """Magnitudes next to where the scale doubles, values on and beside the
    middle of two 8-bit values, zeros, and the ends of f32's range."""
    top = torch.finfo(fp8).max
    one = torch.tensor(1.0)
    peaks = [top, float(torch.nextafter(one * top, one * 1e30)), float(torch.nextafter(one * top, one * 0)), 1.75, 1.7500001,
             2.0 ** -110 * top, 2.0 ** -118 * top, 2.0 ** -119 * top, 1e-44, 0.0, 3.3e38, 2.0 ** 120]
    x = torch.zeros(len(peaks), 256)
    codes = torch.arange(0, 120, dtype=torch.uint8).view(fp8).float()
    mid = (codes[1:] + codes[:-1]) / 2
    for i, p in enumerate(peaks):
        s = 2.0 ** math.floor(math.log2(p / top)) if p > 1e-40 else 1.0
        x[i, :mid.numel()] = torch.where(mid * s <= p, mid * s, 0.0) * (1 if i % 2 else -1)
        x[i, 127] = p
        x[i, 128:247] = torch.nextafter(x[i, :119], torch.zeros(119))
        x[i, 255] = -p
    if tile:
        for row in x:
            check_quantised(row.reshape(2, 128).cuda(), True, fp8)
    else:
        check_quantised(x.cuda(), False, fp8)


@pytest.mark.parametrize("tile", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_quantise_spreads_what_is_not_finite_over_its_block_only(bad, tile):
    x = tokens(200, 300, F32)
    x[5, 140] = bad
    check_quantised(x, tile)


@pytest.mark.parametrize("want_q,want_t", [(True, False), (False, True), (False, False)])
@pytest.mark.parametrize("tile", [False, True])
def test_quantise_one_side_only(want_q, want_t, tile):
    x = tokens(150, 200)
    both = ssd.ssd_block_quantize(x, tile=tile, want_t=True)
    one = ssd.ssd_block_quantize(x, tile=tile, want_q=want_q, want_t=want_t)
    for a, b, wanted in zip(one, both, (want_q, want_q, want_t, want_t)):
        assert a is None if not wanted else torch.equal(a.float(), b.float())


@pytest.mark.parametrize("rows,cols", [(0, 5), (5, 0), (0, 0)])
def test_quantise_nothing(rows, cols):
    q, s, qt, st = ssd.ssd_block_quantize(torch.empty(rows, cols, device="cuda"), want_t=True)
    assert q.shape == (rows, cols) and qt.shape == (cols, rows)
    assert s.shape == (rows, -(-cols // 128)) and st.shape == (cols, -(-rows // 128))


# ----------------------------------------------------------------- products

def operand(rows, cols, tile, seed, fp8=E4, layout="blocks"):
    """A matrix with scales that are no powers of two, in another memory order."""
    q, s, _, _ = ssd.ssd_block_quantize(tokens(rows, cols, F32, seed), tile=tile, fp8=fp8)
    s = s * (1 + torch.rand(s.shape, generator=torch.Generator().manual_seed(seed)).cuda())
    if layout == "rows":
        s = s.contiguous()
    elif layout == "spread":
        wide = torch.zeros(3 * s.shape[0], 2 * s.shape[1], device="cuda")
        wide[::3, ::2] = s
        s = wide[::3, ::2]
    return q, s, blocks.values(np64(q), np64(s))


SIZES = [  # few rows (each width of the tile), blocks that end inside, one of everything, many tiles
    (1, 1, 1), (1, 200, 700), (3, 1, 129), (8, 300, 2000), (33, 130, 257), (65, 500, 128), (128, 129, 1500), (129, 128, 640),
    (200, 31, 500), (257, 64, 1000), (300, 33, 130), (1000, 127, 300), (400, 400, 2100), (1, 5000, 300), (130, 130, 5000),
]
LARGE = [(2000, 2056, 300), (1999, 2051, 257), (5000, 1300, 130)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("tile_a,tile_b", [(False, True), (False, False), (True, False), (True, True)])
def test_matmul(m, n, k, out, tile_a, tile_b):
    a, sa, va = operand(m, k, tile_a, 1)
    b, sb, vb = operand(n, k, tile_b, 2)
    check_product(ssd.ssd_block_matmul(a, sa, b, sb, out_dtype=out), va, vb)


@pytest.mark.parametrize("m,n,k", LARGE)
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("tile", [False, True])
def test_matmul_many_tiles(m, n, k, out, tile):
    a, sa, va = operand(m, k, False, 3)
    b, sb, vb = operand(n, k, tile, 4)
    check_product(ssd.ssd_block_matmul(a, sa, b, sb, out_dtype=out), va, vb)


@pytest.mark.parametrize("n", [29, 30, 33, 34, 36, 40, 50, 62, 63, 64, 90, 94, 100, 126, 127, 130, 186, 250, 333, 500])
@pytest.mark.parametrize("m,k", [(150, 200), (700, 1500), (8071, 300)])
@pytest.mark.parametrize("out", [BF, F32])
def test_matmul_widths(m, n, k, out):
    """Rows of the output on every kind of boundary, and tiles of every width."""
    a, sa, va = operand(m, k, False, 1)
    b, sb, vb = operand(n, k, True, 2)
    y = torch.full((m, n), float("nan"), dtype=out, device="cuda")
    ssd.ssd_block_matmul(a, sa, b, sb, out_dtype=out, out=y)
    check_product(y, va, vb)


@pytest.mark.parametrize("m,n,k", [(40, 300, 900), (300, 300, 900), (2000, 2056, 300)])
@pytest.mark.parametrize("ta,tb", [(E4, E5), (E5, E4), (E5, E5)])
def test_matmul_types(m, n, k, ta, tb):
    a, sa, va = operand(m, k, False, 5, ta)
    b, sb, vb = operand(n, k, True, 6, tb)
    check_product(ssd.ssd_block_matmul(a, sa, b, sb, out_dtype=F32), va, vb)


@pytest.mark.parametrize("layout", ["rows", "spread"])
@pytest.mark.parametrize("m,n,k", [(40, 300, 900), (300, 300, 900), (2000, 2056, 300)])
@pytest.mark.parametrize("tile", [False, True])
def test_matmul_scale_layouts(m, n, k, layout, tile):
    a, sa, va = operand(m, k, False, 7, layout=layout)
    b, sb, vb = operand(n, k, tile, 8, layout=layout)
    check_product(ssd.ssd_block_matmul(a, sa, b, sb, out_dtype=F32), va, vb)


def test_matmul_one_scale_for_all():
    a, _, _ = operand(70, 300, False, 9)
    b, _, _ = operand(90, 300, True, 10)
    one = torch.tensor([[0.25]], device="cuda")
    got = ssd.ssd_block_matmul(a, one.expand(70, 3), b, one.expand(1, 3), out_dtype=F32)
    check_product(got, np64(a) * 0.25, np64(b) * 0.25)


@pytest.mark.parametrize("m,n,k", [(0, 5, 300), (5, 0, 300), (7, 9, 0)])
def test_matmul_nothing(m, n, k):
    def empty(rows):
        return torch.zeros(rows, -(-k // 16) * 16, dtype=torch.uint8, device="cuda")[:, :k].view(E4), \
            torch.ones(rows, -(-k // 128), device="cuda")
    out = torch.full((m, n), 3.0, device="cuda")
    got = ssd.ssd_block_matmul(*empty(m), *empty(n), out_dtype=F32, out=out)
    assert got is not None and out.shape == (m, n) and not out.any()


@pytest.mark.parametrize("m,n,k", [(20, 300, 900), (300, 300, 900), (2000, 2056, 300)])
def test_matmul_keeps_nan_to_its_rows_and_columns(m, n, k):
    x, y = tokens(m, k, F32, 1), tokens(n, k, F32, 2)
    x[m // 2, k - 1] = float("nan")
    y[n // 3, 5] = float("inf")
    a, b = ssd.ssd_block_quantize(x), ssd.ssd_block_quantize(y)
    got = ssd.ssd_block_matmul(a[0], a[1], b[0], b[1])
    want = torch.zeros(m, n, dtype=torch.bool, device="cuda")
    want[m // 2], want[:, n // 3] = True, True
    assert torch.equal(torch.isnan(got), want)


@pytest.mark.parametrize("m,n,k", [(20, 301, 900), (300, 301, 900), (2000, 2051, 300), (2000, 2056, 300)])
def test_matmul_writes_its_output_only_and_repeats(m, n, k):
    a, sa, _ = operand(m, k, False, 1)
    b, sb, _ = operand(n, k, False, 2)
    buf = torch.full((m * n + 512,), -5.0, dtype=BF, device="cuda")
    out = buf[256:256 + m * n].view(m, n)
    assert ssd.ssd_block_matmul(a, sa, b, sb, out=out) is not None
    assert bool((buf[:256] == -5).all()) and bool((buf[256 + m * n:] == -5).all())
    odd = buf[255:255 + m * n].view(m, n)  # off the vectors' boundaries
    first = out.clone()
    ssd.ssd_block_matmul(a, sa, b, sb, out=odd)
    assert torch.equal(odd, first)


# --------------------------------------------------------------- projection

PROJECTIONS = [(1, 64, 200), (8, 260, 500), (37, 129, 1), (128, 1000, 130), (300, 517, 333), (1500, 260, 2100)]


@pytest.mark.parametrize("t,k,n", PROJECTIONS)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("keep", [False, True])
def test_projection_and_gradients(t, k, n, dtype, keep):
    x, w = tokens(t, k, dtype, 1, row=k + 24), tokens(n, k, F32, 2) / math.sqrt(k)
    dy = tokens(t, n, dtype, 3)
    q, s, qt, st = ssd.ssd_block_quantize(w, tile=True, want_t=True)
    y, x_t, x_t_scale = ssd.ssd_projection(x, q, s, return_kept=keep)
    vw, vx = blocks.values(np64(q), np64(s)), blocks.values(*blocks.quantise(np64(x)))
    check_product(y, vx, vw)
    if not keep:
        assert x_t is None and x_t_scale is None
        return
    g = ssd.ssd_projection_bwd(dy, qt, st, x_t, x_t_scale)
    vdy, vdyt, vxt = (blocks.values(*blocks.quantise(v)) for v in (np64(dy), np64(dy).T, np64(x).T))
    check_product(g["dx"], vdy, vw.T)
    check_product(g["dweight"], vdyt, vxt)
    assert g["dx"].dtype == dtype and g["dweight"].dtype == F32
    # one of the two alone is the same
    only = ssd.ssd_projection_bwd(dy, qt, st)
    assert only["dweight"] is None and torch.equal(only["dx"], g["dx"])
    only = ssd.ssd_projection_bwd(dy, x_t=x_t, x_t_scale=x_t_scale)
    assert only["dx"] is None and torch.equal(only["dweight"], g["dweight"])


def test_projection_shapes():
    x = tokens(24, 64).view(2, 3, 4, 64)
    q, s, qt, st = ssd.ssd_block_quantize(tokens(40, 64, F32, 2), tile=True, want_t=True)
    y, x_t, xs = ssd.ssd_projection(x, q, s, return_kept=True)
    assert y.shape == (2, 3, 4, 40) and x_t.shape == (64, 24) and xs.shape == (64, 1)
    flat = ssd.ssd_projection(x.view(24, 64), q, s)[0]
    assert torch.equal(y.view(24, 40), flat)
    assert ssd.ssd_projection_bwd(y, qt, st, x_t, xs)["dx"].shape == x.shape
    one = ssd.ssd_projection(x[0, 0, 0], q, s)[0]
    assert torch.equal(one, flat[0])


@pytest.mark.parametrize("shape", [(0, 64), (2, 0, 64)])
def test_projection_of_no_tokens(shape):
    x = torch.empty(shape, dtype=BF, device="cuda")
    q, s, qt, st = ssd.ssd_block_quantize(tokens(40, 64, F32, 2), tile=True, want_t=True)
    y, x_t, xs = ssd.ssd_projection(x, q, s, return_kept=True)
    g = ssd.ssd_projection_bwd(y, qt, st, x_t, xs)
    assert y.shape == shape[:-1] + (40,) and g["dx"].shape == shape
    assert g["dweight"].shape == (40, 64) and not g["dweight"].any()


def test_each_token_is_its_own():
    """A token's output does not depend on the tokens beside it, whichever tile
    it falls in (the sums' order goes by the number of tokens)."""
    q, s, _, _ = ssd.ssd_block_quantize(tokens(300, 512, F32, 2), tile=True)
    x = tokens(700, 512, F32, 1)
    every = ssd.ssd_projection(x, q, s)[0]
    for n in (1, 20, 64, 129, 500):
        part = ssd.ssd_projection(x[:n], q, s)[0]
        torch.testing.assert_close(part, every[:n], rtol=2.0 ** -18, atol=float(every.abs().max()) * 2.0 ** -20)


# ------------------------------------------------------------------ autograd

@pytest.mark.parametrize("wdtype", [F32, BF])
def test_autograd(wdtype):
    x, w = tokens(150, 200, BF, 1).requires_grad_(), tokens(90, 200, wdtype, 2).requires_grad_()
    y = ssd.ProjectionFunction.apply(x, w)
    dy = tokens(150, 90, BF, 3)
    dx, dw = torch.autograd.grad(y, (x, w), dy)
    vw = blocks.values(*blocks.quantise(np64(w), tile=True))
    check_product(y, blocks.values(*blocks.quantise(np64(x))), vw)
    vdy, vdyt, vxt = (blocks.values(*blocks.quantise(v)) for v in (np64(dy), np64(dy).T, np64(x).T))
    check_product(dx, vdy, vw.T)
    check_product(dw, vdyt, vxt)
    assert dw.dtype == wdtype
    for i, t in enumerate((x, w)):  # one alone
        args = [v if v is t else v.detach() for v in (x, w)]
        g, = torch.autograd.grad(ssd.ProjectionFunction.apply(*args), t, dy)
        assert torch.equal(g, (dx, dw)[i])
    with torch.no_grad():
        assert torch.equal(ssd.ProjectionFunction.apply(x, w), y)


def test_gradients_by_differences():
    """Values that 8 bits hold exactly before and after the step: the output is
    then linear in them and a difference is the gradient."""
    g = torch.Generator().manual_seed(0)

    def whole(*shape):
        return torch.randint(-4, 5, shape, generator=g).float().cuda()
    x, w, dy = whole(20, 70).requires_grad_(), whole(30, 70).requires_grad_(), whole(20, 30)
    dx, dw = torch.autograd.grad(ssd.ProjectionFunction.apply(x, w), (x, w), dy)

    def loss(x, w):
        return float((ssd.ProjectionFunction.apply(x, w).detach().double() * dy.double()).sum())
    with torch.no_grad():
        for t, d in ((x, dx), (w, dw)):
            for i, j in ((0, 0), (7, 69), (19, 33)):
                up, down = t.clone(), t.clone()
                up[i, j] += 1
                down[i, j] -= 1
                a, b = ((up, w), (down, w)) if t is x else ((x, up), (x, down))
                assert (loss(*a) - loss(*b)) / 2 == float(d[i, j])


def test_second_order_is_refused():
    x, w = tokens(5, 20, F32).requires_grad_(), tokens(7, 20, F32).requires_grad_()
    g, = torch.autograd.grad(ssd.ProjectionFunction.apply(x, w).square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="second-order"):
        g.sum().backward()


# ------------------------------------------- streams, workspaces and graphs

def test_streams_and_a_shared_workspace():
    q, s, qt, st = ssd.ssd_block_quantize(tokens(500, 300, F32, 2), tile=True, want_t=True)
    xs = [tokens(n, 300, BF, n) for n in (5, 200, 900)]
    want = []
    for x in xs:
        y, x_t, sc = ssd.ssd_projection(x, q, s, return_kept=True)
        want.append((y, ssd.ssd_projection_bwd(y, qt, st, x_t, sc)))
    ws, side = ssd.Workspace(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for x, (y0, g0) in zip(xs, want):
        y, x_t, sc = ssd.ssd_projection(x, q, s, return_kept=True, workspace=ws, stream=side)
        g = ssd.ssd_projection_bwd(y, qt, st, x_t, sc, workspace=ws, stream=side)
        side.synchronize()
        assert torch.equal(y, y0) and all(torch.equal(g[k], g0[k]) for k in g)


@pytest.mark.parametrize("t", [8, 200, 2000])
def test_captured_and_replayed(t):
    """Forward and backward in one graph, replayed on other inputs, beside an
    eager graph of the same leaves."""
    x, w = tokens(t, 300, BF, 1).requires_grad_(), (tokens(2100, 300, F32, 2) / 17).requires_grad_()
    eager = ssd.ProjectionFunction.apply(x, w)

    def step():
        xd, wd = x.detach(), w.detach()
        q, s, qt, st = ssd.ssd_block_quantize(wd, tile=True, want_t=True)
        y, x_t, sc = ssd.ssd_projection(xd, q, s, return_kept=True)
        return y, ssd.ssd_projection_bwd(y, qt, st, x_t, sc)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, g = step()
    with torch.no_grad():
        x.copy_(tokens(t, 300, BF, 5))
    graph.replay()
    y1, g1 = step()
    assert torch.equal(y, y1) and all(torch.equal(g[k], g1[k]) for k in g)
    assert not torch.equal(eager.detach(), y1)
    assert ssd.ssd_stream_status() == 0


@pytest.mark.parametrize("t", [8, 100, 2000])
def test_inputs_written_just_before(t):
    """Each call reads what the kernel before it on the stream has written:
    inputs, weights and workspace change from call to call without a pause."""
    w = [tokens(300, 512, F32, i) for i in range(2)]
    x = [tokens(t, 512, BF, 7 + i) for i in range(2)]
    want = [ssd.ssd_projection(x[i], *ssd.ssd_block_quantize(w[i], tile=True)[:2])[0] for i in range(2)]
    torch.cuda.synchronize()
    ws, xb, wb = ssd.Workspace(), torch.empty_like(x[0]), torch.empty_like(w[0])
    got = []
    for i in range(60):
        wb.copy_(w[i % 2])
        q, s, _, _ = ssd.ssd_block_quantize(wb, tile=True)
        xb.copy_(x[i % 2])
        got.append(ssd.ssd_projection(xb, q, s, workspace=ws)[0])
        if i % 3 == 0:  # the weights' kernel last
            q, s, _, _ = ssd.ssd_block_quantize(wb, tile=True)
            got[-1] = ssd.ssd_projection(xb, q, s, workspace=ws)[0]
    assert all(torch.equal(g, want[i % 2]) for i, g in enumerate(got))


def test_two_streams_at_once():
    """Calls of all kinds of tiles beside one another on two streams."""
    cases = []
    for t, k, n in ((5, 700, 900), (60, 300, 1000), (120, 900, 640), (400, 384, 300), (3000, 256, 2100)):
        x, (q, s, _, _) = tokens(t, k, BF, t), ssd.ssd_block_quantize(tokens(n, k, F32, n), tile=True)
        cases.append((x, q, s, ssd.ssd_projection(x, q, s)[0]))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(20):
        for i, st in enumerate(streams):
            for x, q, s, _ in cases[::-1] if i else cases:
                got[i].append(ssd.ssd_projection(x, q, s, stream=st)[0])
    torch.cuda.synchronize()
    for i in range(2):
        order = cases[::-1] if i else cases
        for j, y in enumerate(got[i]):
            assert torch.equal(y, order[j % len(order)][3])
    assert ssd.ssd_stream_status() == 0


def test_offsets_past_32_bits():
    """Matrices of more than 2^32 bytes and outputs of more than 2^31 elements: the
    last rows are those of a small call on them alone."""
    m, k, n = (1 << 20) + 77, 4112, 2056
    x = torch.empty(m, k, dtype=BF, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(0))
    q, s, qt, st = ssd.ssd_block_quantize(x, want_t=True)
    last = ssd.ssd_block_quantize(x[-300:])
    assert torch.equal(q[-300:].float(), last[0].float()) and torch.equal(s[-300:], last[1])
    # the transpose's last row, block by block of 128 tokens
    col = x[:, -1].float()
    pad = torch.nn.functional.pad(col, (0, -m % 128)).view(-1, 128)
    values = (qt[-1].float() * st[-1].repeat_interleave(128)[:m])
    assert bool(((values - col).abs() <= 2.0 ** -4 * pad.abs().amax(1).repeat_interleave(128)[:m]).all())
    assert torch.equal(values[:128], qt[-1, :128].float() * st[-1, 0]) and bool((values != 0).any())
    b, sb, _, _ = ssd.ssd_block_quantize(tokens(n, k, F32, 3), tile=True)
    y = ssd.ssd_block_matmul(q, s, b, sb)
    assert y.numel() > 1 << 31
    for rows in (slice(-300, None), slice(0, 300), slice(m // 2, m // 2 + 300)):
        part = ssd.ssd_block_matmul(q[rows], s[rows], b, sb, out_dtype=F32)
        assert bool(((y[rows].float() - part).abs() <= 2.0 ** -8 * part.abs() + 2.0 ** -14 * float(part.abs().max())).all())
    assert ssd.ssd_stream_status() == 0


@pytest.mark.parametrize("inference", [False, True])
def test_the_transposes_scales_of_tiles_are_the_tiles(inference):
    """One memory and one version for both, in inference mode too."""
    with torch.inference_mode(inference):
        _, s, _, st = ssd.ssd_block_quantize(tokens(300, 200, F32), tile=True, want_t=True)
        assert st.shape == (2, 3) and torch.equal(st, s.t()) and st.data_ptr() == s.data_ptr()
        assert s.is_inference() == st.is_inference() == inference
        s[2, 1] = 7.0
        assert float(st[1, 2]) == 7.0
        if not inference:
            assert st._version == s._version == 1


@pytest.mark.parametrize("rows", list(range(241, 258)))
@pytest.mark.parametrize("wide", [False, True])
def test_quantise_tails(rows, wide):
    """Every number of last rows and columns, with 16 warps a block and with 8."""
    check_quantised(tokens(rows, 13000 if wide else 300 - rows % 17, BF, rows), False)
    check_quantised(tokens(rows, 12996 if wide else rows, F32, rows), True)
