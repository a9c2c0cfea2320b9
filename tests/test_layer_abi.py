"""Refusals of the layer operators' entry points: every class of bad argument
is answered on the host, before any launch (no GPU needed)."""
import ctypes

import pytest

from state_space_sequence_cumsum_gb300 import _lib

INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = (_lib.SSD_ERR_INVALID_ARG, _lib.SSD_ERR_UNSUPPORTED,
                                              _lib.SSD_ERR_ALIGNMENT, _lib.SSD_ERR_WORKSPACE)


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


def conv(lib, dims=(2, 8, 16, 4), row=16, dtype=0, **kw):
    p = dict(zip(("x", "w", "bias", "init", "y", "fin"), ptrs(6)))
    p.update(kw)
    return lib.ssd_causal_conv(p["x"], row, p["w"], p["bias"], p["init"], p["y"], p["fin"],
                               _lib.ssd_conv_dims_t(*dims), 1, dtype, None)


def test_conv_refusals(lib):
    assert conv(lib, dims=(0, 8, 16, 4)) == INVALID
    assert conv(lib, dims=(2, -1, 16, 4)) == INVALID
    assert conv(lib, dims=(2, 8, 0, 4)) == INVALID
    assert conv(lib, dims=(2, 8, 16, 1)) == UNSUPPORTED
    assert conv(lib, dims=(2, 8, 16, 5)) == UNSUPPORTED
    assert conv(lib, dims=(70000, 8, 16, 4)) == UNSUPPORTED
    assert conv(lib, dims=(2, 1 << 41, 16, 4)) == UNSUPPORTED
    assert conv(lib, row=15) == INVALID
    assert conv(lib, dtype=7) == INVALID
    for name in ("x", "w", "y"):
        assert conv(lib, **{name: None}) == INVALID
    p = ptrs(6)
    assert conv(lib, x=at(p[0], 1)) == ALIGNMENT
    assert conv(lib, w=at(p[1], 2)) == ALIGNMENT
    assert conv(lib, y=p[0]) == INVALID                # in place: the window reads what was written
    assert conv(lib, fin=p[3]) == INVALID
    assert conv(lib, y=at(p[0], 2 * (15 * 16 + 15))) == INVALID  # the last element


def test_conv_bwd_and_step_refusals(lib):
    d = _lib.ssd_conv_dims_t(2, 8, 16, 4)
    need = lib.ssd_causal_conv_bwd_workspace_size(d)
    assert need > 0 and need % 256 == 0
    assert lib.ssd_causal_conv_bwd_workspace_size(_lib.ssd_conv_dims_t(2, 8, 16, 9)) == 0

    def bwd(ws, size, row_dy=16, **kw):
        names = ("x", "w", "bias", "init", "dy", "dfinal", "dx", "dw", "db", "dinit")
        p = dict(zip(names, ptrs(10)))
        p.update(kw)
        return lib.ssd_causal_conv_bwd(p["x"], 16, p["w"], p["bias"], p["init"], p["dy"], row_dy, p["dfinal"],
                                       p["dx"], p["dw"], p["db"], p["dinit"], d, 1, 0, ws, size, None)
    ws = ptrs(1, 20)[0]
    assert bwd(None, need) == WORKSPACE
    assert bwd(ws, need - 1) == WORKSPACE
    assert bwd(at(ws, 16), need) == WORKSPACE
    assert bwd(ws, need, row_dy=8) == INVALID
    assert bwd(ws, need, dx=ptrs(10)[4]) == INVALID
    assert bwd(ws, need, dy=None) == INVALID
    p = ptrs(5)

    def step(dims=(2, 1, 16, 4), state=p[2], out=p[2], y=p[3]):
        return lib.ssd_causal_conv_step(p[0], 16, p[1], None, state, out, y, _lib.ssd_conv_dims_t(*dims), 1, 0, None)
    assert step(dims=(2, 2, 16, 4)) == INVALID
    assert step(out=at(p[2], 16)) == INVALID           # partly overlapping states
    assert step(state=None) == INVALID
    assert step(y=p[2]) == INVALID


SCAN_NAMES = ("u", "dt", "A", "B", "C", "D", "z", "bias", "init", "y", "fin", "kept")


def scan(lib, dims=(2, 40, 16, 8, 2), rows=None, dtype=0, ws=None, size=0, **kw):
    p = dict(zip(SCAN_NAMES, ptrs(12)))
    p.update(kw)
    rows = rows or (dims[2], dims[2], dims[2], dims[3] * dims[4], dims[3] * dims[4], dims[2])
    return lib.ssd_selective_scan(*[p[n] for n in SCAN_NAMES], _lib.ssd_scan_dims_t(*dims), _lib.ssd_scan_rows_t(*rows),
                                  1, dtype, ws, size, None)


def test_scan_refusals(lib):
    assert scan(lib, dims=(0, 40, 16, 8, 2)) == INVALID
    assert scan(lib, dims=(2, 40, 16, 8, 3)) == INVALID
    assert scan(lib, dims=(2, 40, 16, 65, 2)) == UNSUPPORTED
    assert scan(lib, dims=(70000, 40, 16, 8, 2)) == UNSUPPORTED
    assert scan(lib, rows=(15, 16, 16, 16, 16, 16)) == INVALID
    assert scan(lib, rows=(16, 16, 16, 15, 16, 16)) == INVALID
    assert scan(lib, rows=(16, 16, 3, 16, 16, 16)) == INVALID
    assert scan(lib, dtype=3) == INVALID
    for name in ("u", "dt", "A", "B", "C", "y"):
        assert scan(lib, **{name: None}) == INVALID
    p = dict(zip(SCAN_NAMES, ptrs(12)))
    assert scan(lib, A=at(p["A"], 2)) == ALIGNMENT
    assert scan(lib, z=at(p["z"], 1)) == ALIGNMENT
    assert scan(lib, y=p["u"]) == INVALID
    assert scan(lib, fin=at(p["init"], 64)) == INVALID     # in place only as a whole
    assert scan(lib, kept=p["fin"]) == INVALID
    long = (1, 4096, 16, 8, 1)
    need = lib.ssd_selective_scan_workspace_size(_lib.ssd_scan_dims_t(*long))
    assert need > 0 and need % 256 == 0                    # few channels, many tokens: segments
    ws = ptrs(1, 30)[0]
    assert scan(lib, dims=long) == WORKSPACE
    assert scan(lib, dims=long, ws=ws, size=need - 1) == WORKSPACE
    assert scan(lib, dims=long, ws=at(ws, 8), size=need) == WORKSPACE
    assert scan(lib, dims=long, ws=p["u"], size=need) == INVALID


def test_scan_bwd_and_step_refusals(lib):
    dims = (2, 40, 16, 8, 2)
    d, r = _lib.ssd_scan_dims_t(*dims), _lib.ssd_scan_rows_t(16, 16, 16, 16, 16, 16)
    names = ("u", "dt", "A", "B", "C", "D", "z", "bias", "init", "dy", "dfin", "kept", "du", "ddt", "dA", "dB", "dC",
             "dD", "dz", "db", "dinit")
    need = lib.ssd_selective_scan_bwd_workspace_size(d, 1)
    assert lib.ssd_selective_scan_bwd_workspace_size(d, 0) > need > 0
    ws = ptrs(1, 60)[0]

    def bwd(ws=ws, size=need, rows=r, **kw):
        p = dict(zip(names, ptrs(21)))
        p.update(kw)
        return lib.ssd_selective_scan_bwd(*[p[n] for n in names], d, rows, 1, 0, ws, size, None)
    assert bwd(ws=None) == WORKSPACE
    assert bwd(size=need - 256) == WORKSPACE
    assert bwd(kept=None) == WORKSPACE                     # the recomputed states need room
    assert bwd(z=None) == INVALID                          # dz without z
    assert bwd(D=None) == INVALID
    assert bwd(dz=None) == INVALID                         # z without dz
    assert bwd(du=None) == INVALID
    assert bwd(dB=dict(zip(names, ptrs(21)))["dC"]) == INVALID
    assert bwd(rows=_lib.ssd_scan_rows_t(16, 16, 16, 16, 16, 8)) == INVALID
    p = ptrs(11)

    def step(dims=(2, 1, 16, 8, 2), state=p[8], out=p[8]):
        return lib.ssd_selective_scan_step(*p[:8], state, out, p[9], _lib.ssd_scan_dims_t(*dims), r, 1, 0, None)
    assert step(dims=(2, 2, 16, 8, 2)) == INVALID
    assert step(out=at(p[8], 4)) == INVALID
    assert step(out=None) == INVALID


def test_block_norm_refusals(lib):
    names = ("y", "res", "w", "pw", "gate", "out", "res_out")

    def norm(tokens=6, dim=16, rows=3, eps=1e-5, dtype=0, rdtype=1, **kw):
        p = dict(zip(names, ptrs(7)))
        p.update(kw)
        return lib.ssd_block_norm(*[p[n] for n in names], tokens, dim, rows, 1.0, eps, dtype, rdtype, None)
    p = dict(zip(names, ptrs(7)))
    assert norm(tokens=-1) == INVALID
    assert norm(dim=0) == INVALID
    assert norm(rows=4) == INVALID                         # 6 tokens, 4 gate rows
    assert norm(rows=0) == INVALID                         # a gate without rows
    assert norm(gate=None) == INVALID                      # rows without a gate
    assert norm(eps=-1.0) == INVALID
    assert norm(eps=float("nan")) == INVALID
    assert norm(dim=32769) == UNSUPPORTED
    assert norm(dtype=1, rdtype=0) == INVALID              # a residual narrower than the block's output
    assert norm(w=None) == INVALID
    assert norm(y=at(p["y"], 1)) == ALIGNMENT
    assert norm(out=p["y"]) == INVALID
    assert norm(res_out=at(p["res"], 4)) == INVALID
    need = lib.ssd_block_norm_bwd_workspace_size(6, 16, 3)
    assert need > 0

    def bwd(ws, size, **kw):
        n2 = ("y", "r", "w", "pw", "gate", "dout", "dr", "dy", "dres", "dw", "dpw", "dg")
        q = dict(zip(n2, ptrs(12)))
        q.update(kw)
        return lib.ssd_block_norm_bwd(*[q[n] for n in n2], 6, 16, 3, 1.0, 1e-5, 0, 1, ws, size, None)
    ws = ptrs(1, 40)[0]
    assert bwd(None, need) == WORKSPACE
    assert bwd(ws, need - 1) == WORKSPACE
    assert bwd(ws, need, dpw=None) == INVALID
    assert bwd(ws, need, dg=None) == INVALID
    assert bwd(ws, need, dw=None) == INVALID
    assert bwd(ws, need, dy=ptrs(12)[5]) == INVALID


def test_binding_refusals():
    torch = pytest.importorskip("torch")
    import state_space_sequence_cumsum_gb300 as ssd
    x, w = torch.zeros(1, 4, 8), torch.zeros(8, 4)
    A, m = torch.zeros(8, 4), torch.zeros(1, 4, 4)

    def refused(error, match, call, *args, **kw):
        with pytest.raises(error, match=match):
            call(*args, **kw)
    refused(ValueError, "CUDA tensors", ssd.ssd_causal_conv, x, w)
    refused(ValueError, "weight must be", ssd.ssd_causal_conv, x, torch.zeros(7, 4))
    refused(ValueError, "activation", ssd.ssd_causal_conv, x, w, activation="relu")
    refused(TypeError, "bfloat16 or float32", ssd.ssd_causal_conv, x.half(), w)
    refused(TypeError, "weight must be", ssd.ssd_causal_conv, x, w.double())
    refused(TypeError, "x must be a tensor", ssd.ssd_causal_conv, None, w)
    refused(ValueError, "last dimension", ssd.ssd_causal_conv,
            x.transpose(1, 2).contiguous().transpose(1, 2), w)
    refused(ValueError, "evenly spaced", ssd.ssd_causal_conv, torch.zeros(2, 8, 8)[:, ::3], w)
    refused(ValueError, "rows overlap", ssd.ssd_causal_conv, torch.zeros(1, 1, 8).expand(1, 4, 8), w)
    refused(ValueError, "initial_state must be", ssd.ssd_causal_conv, x, w, initial_state=torch.zeros(1, 2, 8))
    refused(ValueError, "C must be", ssd.ssd_selective_scan, x, x, A, m, torch.zeros(1, 4, 5))
    refused(ValueError, "multiple of the groups", ssd.ssd_selective_scan, x, x, A, torch.zeros(1, 4, 3, 4),
            torch.zeros(1, 4, 3, 4))
    refused(ValueError, "dt must be", ssd.ssd_selective_scan, x, x[:, :2], A, m, m)
    refused(TypeError, "initial_state must be", ssd.ssd_selective_scan, x, x, A, m, m,
            initial_state=torch.zeros(1, 8, 4, dtype=torch.bfloat16))
    refused(ValueError, "state must be", ssd.ssd_selective_scan_step, x[:, 0], x[:, 0], A, m[:, 0], m[:, 0], None,
            torch.zeros(1, 8, 5))
    refused(ValueError, "weight must be", ssd.ssd_block_norm, x, x, torch.zeros(7))
    refused(ValueError, "gate's rows", ssd.ssd_block_norm, x, x, torch.zeros(8), gate=torch.zeros(3, 8))
    refused(ValueError, "residual must be", ssd.ssd_block_norm, x, torch.zeros(1, 4, 9), torch.zeros(8))
    refused(ValueError, "y must be contiguous", ssd.ssd_block_norm, x[:, ::2], x, torch.zeros(8))
    refused(TypeError, "residual must be", ssd.ssd_block_norm, x, None, torch.zeros(8),
            residual_dtype=torch.bfloat16)
