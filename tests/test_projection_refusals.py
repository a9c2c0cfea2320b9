"""Refusals of the 8-bit projections' and the optimiser's entry points: every
class of bad argument is answered on the host, before any launch (no GPU
needed)."""
import ctypes

import pytest
import torch

import state_space_sequence_cumsum_gb300 as ssd
from state_space_sequence_cumsum_gb300 import _lib

OK, INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = (_lib.SSD_OK, _lib.SSD_ERR_INVALID_ARG, _lib.SSD_ERR_UNSUPPORTED,
                                                  _lib.SSD_ERR_ALIGNMENT, _lib.SSD_ERR_WORKSPACE)
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def lib():
    lib = _lib.load()
    before = lib.ssd_launch_count()
    yield lib
    assert lib.ssd_launch_count() == before


def ptrs(n, start=1):
    """n addresses far apart (never dereferenced: the calls are refused)."""
    return [ctypes.c_void_p((start + i) << 40) for i in range(n)]


def at(p, off):
    return ctypes.c_void_p(p.value + off)


def quantize(lib, rows=200, cols=300, row=300, dtype=0, tile=0, type=0, row_q=304, scale_ld=200, row_qt=208,
             scale_t_ld=300, **kw):
    p = dict(zip(("x", "q", "scale", "q_t", "scale_t"), ptrs(5)), **kw)
    return lib.ssd_block_quantize(p["x"], row, rows, cols, dtype, tile, type, p["q"], row_q, p["scale"], scale_ld,
                                  p["q_t"], row_qt, p["scale_t"], scale_t_ld, None)


def test_quantize_refusals(lib):
    p = ptrs(5)
    assert quantize(lib, rows=-1) == INVALID
    assert quantize(lib, row=299) == INVALID
    assert quantize(lib, dtype=2) == INVALID
    assert quantize(lib, type=2) == INVALID
    assert quantize(lib, x=None) == INVALID
    assert quantize(lib, scale=None) == INVALID
    assert quantize(lib, scale_t=None) == INVALID
    assert quantize(lib, q=None) == INVALID                    # its scale is given
    assert quantize(lib, tile=1) == INVALID                    # one set of scales
    assert quantize(lib, tile=1, scale_t=None, scale_ld=2) == INVALID
    assert quantize(lib, scale_ld=199) == INVALID
    assert quantize(lib, scale_t_ld=299) == INVALID
    assert quantize(lib, row_q=299) == INVALID
    assert quantize(lib, row_q=308) == ALIGNMENT
    assert quantize(lib, row_qt=204) == ALIGNMENT
    assert quantize(lib, q=at(p[1], 8)) == ALIGNMENT
    assert quantize(lib, q_t=at(p[3], 4)) == ALIGNMENT
    assert quantize(lib, x=at(p[0], 1)) == ALIGNMENT
    assert quantize(lib, scale=at(p[2], 2)) == ALIGNMENT
    assert quantize(lib, q=p[0]) == INVALID                    # in place
    assert quantize(lib, q_t=at(p[1], 199 * 304 + 288)) == INVALID  # q's last row
    assert quantize(lib, scale_t=p[2]) == INVALID
    assert quantize(lib, rows=1 << 31) == UNSUPPORTED
    assert quantize(lib, rows=1 << 22, cols=1 << 22, row=1 << 22, row_q=1 << 22, row_qt=1 << 22, scale_ld=1 << 22,
                    scale_t_ld=1 << 22) == UNSUPPORTED
    assert quantize(lib, rows=0) == OK and quantize(lib, cols=0) == OK  # nothing to do
    assert quantize(lib, q=None, scale=None, q_t=None, scale_t=None) == OK


def matrix(p, row=304, scale_row=1, scale_block=200, tile=0, type=0, **kw):
    a = {"values": p[0], "scales": p[1], **kw}
    return _lib.ssd_block_matrix_t(a["values"], a["scales"], row, scale_row, scale_block, tile, type)


def matmul(lib, m=200, n=500, k=300, out_dtype=0, out=None, a=None, b=None):
    p = ptrs(5)
    a, b = (matrix(p[2 * i:2 * i + 2], **(given or {})) for i, given in enumerate((a, b)))
    return lib.ssd_block_matmul(a, b, p[4] if out is None else out, m, n, k, out_dtype, None)


def test_matmul_refusals(lib):
    p = ptrs(5)
    b = dict(scale_block=500)
    assert matmul(lib, m=-1, b=b) == INVALID
    assert matmul(lib, k=-1, b=b) == INVALID
    assert matmul(lib, out_dtype=3, b=b) == INVALID
    assert matmul(lib, m=1 << 31, b=b) == UNSUPPORTED
    assert matmul(lib, m=1 << 30, n=1 << 30, b=b) == UNSUPPORTED
    assert matmul(lib, out=ctypes.c_void_p(0), b=b) == INVALID
    assert matmul(lib, out=at(p[4], 1), b=b) == ALIGNMENT
    for which in ("a", "b"):
        def bad(**kw):
            return matmul(lib, **{"a": dict(scale_block=200), "b": dict(scale_block=500), which: kw})
        assert bad(values=None) == INVALID
        assert bad(scales=None) == INVALID
        assert bad(type=2) == INVALID
        assert bad(row=288) == INVALID
        assert bad(row=312) == ALIGNMENT
        assert bad(values=at(p[0], 8)) == ALIGNMENT
        assert bad(scales=at(p[1], 2)) == ALIGNMENT
        assert bad(scale_row=-1) == INVALID
        assert bad(scale_block=-1) == INVALID
        assert bad(scale_row=1 << 40) == UNSUPPORTED
        assert bad(values=p[4]) == INVALID                     # the output
        assert bad(scales=at(p[4], 200 * 500 * 2 - 4)) == INVALID
    assert matmul(lib, m=0, b=b) == OK and matmul(lib, n=0) == OK


def test_projection_refusals(lib):
    need = lib.ssd_projection_workspace_size(200, 300)
    assert need > 0 and need % 256 == 0 and lib.ssd_projection_workspace_size(-1, 300) == 0
    names = ("x", "w", "s", "y", "x_t", "x_t_scale", "ws")

    def call(row=300, dtype=0, row_xt=208, ld=300, size=need, tokens=200, weight=None, **kw):
        p = dict(zip(names, ptrs(7)), **kw)
        w = matrix([p["w"], p["s"]], **(weight or dict(scale_row=3, scale_block=1, tile=1)))
        return lib.ssd_projection(p["x"], row, w, p["y"], p["x_t"], row_xt, p["x_t_scale"], ld, tokens, 300, 500, dtype,
                                  p["ws"], size, None)
    p = dict(zip(names, ptrs(7)))
    assert call(row=299) == INVALID
    assert call(dtype=5) == INVALID
    assert call(tokens=-1) == INVALID
    for name in ("x", "w", "s", "y", "x_t_scale"):
        assert call(**{name: None}) == INVALID
    assert call(x_t=None) == INVALID                           # its scales are given
    assert call(row_xt=192) == INVALID
    assert call(row_xt=204) == ALIGNMENT
    assert call(ld=299) == INVALID
    assert call(ws=None) == WORKSPACE
    assert call(size=need - 1) == WORKSPACE
    assert call(ws=at(p["ws"], 128)) == WORKSPACE
    assert call(y=p["x"]) == INVALID
    assert call(ws=p["w"]) == INVALID
    assert call(weight=dict(row=296)) == INVALID

    bneed = lib.ssd_projection_bwd_workspace_size(200, 500, 1, 1)
    halves = [lib.ssd_projection_bwd_workspace_size(200, 500, i, 1 - i) for i in (0, 1)]
    assert bneed == sum(halves) and lib.ssd_projection_bwd_workspace_size(200, 500, 0, 0) == 0
    bnames = ("dy", "w", "s", "x", "xs", "dx", "dw", "ws")

    def bwd(row=500, size=bneed, weight=None, kept=None, **kw):
        p = dict(zip(bnames, ptrs(8)), **kw)
        mw = matrix([p["w"], p["s"]], **(weight or dict(row=512, scale_row=1, scale_block=3, tile=1)))
        mx = matrix([p["x"], p["xs"]], **(kept or dict(row=208, scale_block=300)))
        return lib.ssd_projection_bwd(p["dy"], row, mw, mx, p["dx"], p["dw"], 200, 300, 500, 0, p["ws"], size, None)
    p = dict(zip(bnames, ptrs(8)))
    assert bwd(row=499) == INVALID
    for name in ("dy", "w", "s", "x", "xs"):
        assert bwd(**{name: None}) == INVALID
    assert bwd(ws=None) == WORKSPACE and bwd(size=bneed - 1) == WORKSPACE
    assert bwd(dx=None, size=halves[0] - 1) == WORKSPACE
    assert bwd(dw=p["dx"]) == INVALID
    assert bwd(weight=dict(row=504)) == ALIGNMENT and bwd(kept=dict(row=204)) == ALIGNMENT
    assert bwd(dx=None, dw=None, dy=None, size=0, ws=None) == OK


def adamw(lib, count=2, bits=32, p_dtype=1, g_dtype=1, n=(1000, 7), lr=0.1, b1=0.9, b2=0.99, eps=1e-8, wd=0.0, step=1,
          lr_device=None, step_device=None, scale_device=None, change=()):
    tensors = (_lib.ssd_adamw_tensor_t * 2)()
    for i in range(2):
        p = ptrs(6, 1 + 6 * i)
        tensors[i] = _lib.ssd_adamw_tensor_t(*p[:4], p[4] if bits == 8 else None, p[5] if bits == 8 else None, n[i])
    for i, name, value in change:
        setattr(tensors[i], name, value)
    args = _lib.ssd_adamw_t(lr, b1, b2, eps, wd, step, 1.0, lr_device, step_device, scale_device)
    return lib.ssd_adamw_step(tensors, count, args, bits, p_dtype, g_dtype, None)


def test_adamw_refusals(lib):
    nan = float("nan")
    for kw in (dict(count=-1), dict(bits=16), dict(p_dtype=2), dict(g_dtype=2), dict(lr=-1.0), dict(lr=nan), dict(b1=1.0),
               dict(b1=-0.1), dict(b2=1.0), dict(b2=nan), dict(eps=-1.0), dict(wd=-1.0), dict(wd=nan), dict(step=0),
               dict(n=(-1, 7))):
        assert adamw(lib, **kw) == INVALID, kw
    assert adamw(lib, n=(1 << 41, 7)) == UNSUPPORTED
    assert lib.ssd_adamw_step(None, 1, _lib.ssd_adamw_t(0.1, 0.9, 0.9, 0, 0, 1, 1.0), 32, 1, 1, None) == INVALID
    p, q = ptrs(6), ptrs(6, 7)
    for bits in (32, 8):
        for name in ("p", "g", "m", "v") + (("m_scale", "v_scale") if bits == 8 else ()):
            assert adamw(lib, bits=bits, change=[(1, name, None)]) == INVALID
    assert adamw(lib, change=[(0, "p", p[0].value + 2)]) == ALIGNMENT
    assert adamw(lib, bits=8, change=[(0, "m_scale", p[4].value + 1)]) == ALIGNMENT
    assert adamw(lib, lr_device=p[0].value + 2) == ALIGNMENT
    assert adamw(lib, step_device=(1 << 50) + 4) == ALIGNMENT
    assert adamw(lib, change=[(1, "p", p[0].value)]) == INVALID             # one tensor twice
    assert adamw(lib, change=[(1, "p", p[0].value + 4 * 999)]) == INVALID   # the last element
    assert adamw(lib, change=[(1, "g", p[2].value)]) == INVALID             # reads what is written
    assert adamw(lib, bits=8, change=[(1, "v_scale", p[4].value + 12)]) == INVALID
    assert adamw(lib, scale_device=q[1].value, change=[(1, "p", q[1].value)]) == INVALID


# ------------------------------------------------------------ Python calls

def mat(rows, cols, row=None, dtype=F8):
    row = -(-cols // 16) * 16 if row is None else row
    return torch.zeros(rows, row, dtype=torch.uint8)[:, :cols].view(dtype)


def scales(rows, cols, tile=False):
    return torch.ones(-(-rows // 128) if tile else rows, -(-cols // 128))


def test_python_refusals_of_the_products():
    x = torch.zeros(4, 40)
    with pytest.raises(TypeError, match="fp8 must be"):
        ssd.ssd_block_quantize(x, fp8=torch.float16)
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        ssd.ssd_block_quantize(x.half())
    with pytest.raises(ValueError, match=r"x must be \[rows, cols\]"):
        ssd.ssd_block_quantize(x[0])
    with pytest.raises(ValueError, match="last dimension must be contiguous"):
        ssd.ssd_block_quantize(x.t())
    with pytest.raises(ValueError, match="CUDA tensors"):
        ssd.ssd_block_quantize(x)
    a, sa, b, sb = mat(4, 40), scales(4, 40), mat(6, 40), scales(6, 40, True)
    with pytest.raises(TypeError, match="out_dtype"):
        ssd.ssd_block_matmul(a, sa, b, sb, out_dtype=torch.float16)
    with pytest.raises(TypeError, match="a must be float8"):
        ssd.ssd_block_matmul(x, sa, b, sb)
    with pytest.raises(ValueError, match="the scales of b must be"):
        ssd.ssd_block_matmul(a, sa, b, torch.ones(3, 1))
    with pytest.raises(TypeError, match="the scales of a must be Float"):
        ssd.ssd_block_matmul(a, sa.double(), b, sb)
    with pytest.raises(ValueError, match="same k"):
        ssd.ssd_block_matmul(a, sa, mat(6, 41), sb)
    with pytest.raises(ValueError, match="CUDA tensors"):
        ssd.ssd_block_matmul(a, sa, b, sb)
    with pytest.raises(ValueError, match=r"weight must be \[outputs, 39\]"):
        ssd.ssd_projection(x[:, :39].contiguous(), b, sb)
    with pytest.raises(ValueError, match=r"weight_t must be \[inputs, 40\]"):
        ssd.ssd_projection_bwd(x, mat(7, 41), scales(7, 41, True))
    with pytest.raises(ValueError, match=r"x_t must be \[inputs, 4\]"):
        ssd.ssd_projection_bwd(x, mat(7, 40), scales(7, 40, True), mat(8, 4), scales(8, 4))
    with pytest.raises(TypeError, match="weight_t_scale must be a tensor"):
        ssd.ssd_projection_bwd(x, mat(7, 40))


def test_python_refusals_of_the_step():
    p = [torch.zeros(300), torch.zeros(4, 5)]
    call = ssd.ssd_adamw_step
    with pytest.raises(ValueError, match="must be as many"):
        call(p, p[:1], p, p, 1)
    with pytest.raises(TypeError, match="list or tuple"):
        call(torch.zeros(2, 3), p, p, p, 1)
    with pytest.raises(TypeError, match="must be a tensor"):
        call(p, [p[0], None], p, p, 1)
    with pytest.raises(ValueError, match="grads must be"):
        call(p, [p[0], torch.zeros(5, 4)], p, p, 1)
    with pytest.raises(TypeError, match="params must be"):
        call([p[0], p[1].bfloat16()], p, p, p, 1)
    with pytest.raises(ValueError, match="must be contiguous"):
        call([p[0], torch.zeros(5, 4).t()], p, p, p, 1)
    with pytest.raises(ValueError, match="given together"):
        call(p, p, p, p, 1, m_scales=p)
    q = [t.to(F8) for t in p]
    with pytest.raises(TypeError, match="m must be Float8_e4m3fn"):
        call(p, p, p, q, 1, m_scales=p, v_scales=p)
    with pytest.raises(ValueError, match=r"m_scales must be \[2\]"):
        call(p, p, q, q, 1, m_scales=p, v_scales=p)
    with pytest.raises(ValueError, match="CUDA tensors"):
        call(p, p, p, p, 1)
    call([], [], [], [], 1)  # nothing to do
    for kw in (dict(lr=-1.0), dict(betas=(0.9, 1.0)), dict(state_bits=4), dict(weight_decay=-0.1)):
        with pytest.raises(ValueError):
            ssd.AdamW([torch.zeros(3, requires_grad=True)], **kw)
