"""Calls from two host threads through the C ABI (ctypes lets go of the
interpreter lock): kernels whose shared memory depends on the row's width, on
widths in turn.  Each thread has its own stream and buffers; every call must be
accepted and give what the same call gives alone."""
import ctypes
import threading

import pytest
import torch

from state_space_sequence_cumsum_gb300 import _lib

pytestmark = pytest.mark.gpu


def in_two_threads(calls, rounds=40):
    """calls[i]: thread i's list of (function of a stream, its outputs)."""
    alone = []
    for mine in calls:
        for call, outs in mine:
            assert call(torch.cuda.current_stream()) == 0
            alone.append([o.clone() for o in outs])
    torch.cuda.synchronize()
    bad, gate = [], threading.Barrier(2)

    def work(mine):
        stream = torch.cuda.Stream()
        gate.wait()
        for _ in range(rounds):
            for call, _ in mine:
                status = call(stream)
                if status:
                    bad.append(status)
        stream.synchronize()
    threads = [threading.Thread(target=work, args=(mine,)) for mine in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert bad == []
    got = [outs for mine in calls for _, outs in mine]
    for a, outs in zip(alone, got):
        for x, y in zip(a, outs):
            assert torch.equal(x, y)


def ptr(t):
    return ctypes.c_void_p(t.data_ptr())


def norm_calls(dim, tokens=3):
    lib, f32 = _lib.load(), _lib.SSD_F32
    g = torch.Generator(device="cuda").manual_seed(dim)
    y, res, dout = (torch.randn(tokens, dim, generator=g, device="cuda") for _ in range(3))
    w, pw = (torch.randn(dim, generator=g, device="cuda") for _ in range(2))
    out, rr, dy, dres = (torch.empty_like(y) for _ in range(4))
    dw, dpw = torch.empty_like(w), torch.empty_like(w)
    ws = torch.empty(lib.ssd_block_norm_bwd_workspace_size(tokens, dim, 0), dtype=torch.uint8, device="cuda")

    def forward(s):
        return lib.ssd_block_norm(ptr(y), ptr(res), ptr(w), ptr(pw), None, ptr(out), ptr(rr), tokens, dim, 0, 0.5,
                                  1e-5, f32, f32, ctypes.c_void_p(s.cuda_stream))

    def backward(s):
        return lib.ssd_block_norm_bwd(ptr(y), ptr(res), ptr(w), ptr(pw), None, ptr(dout), None, ptr(dy), ptr(dres),
                                      ptr(dw), ptr(dpw), None, tokens, dim, 0, 0.5, 1e-5, f32, f32, ptr(ws),
                                      ws.numel(), ctypes.c_void_p(s.cuda_stream))
    return [(forward, [out, rr]), (backward, [dy, dres, dw, dpw])]


def test_norms_of_two_widths():
    # backward through rings of 80 and 160 KB, wide rows of 40 to 128 KB both ways
    in_two_threads([norm_calls(2560) + norm_calls(10240) + norm_calls(32768),
                    norm_calls(5120) + norm_calls(12288) + norm_calls(20480)])


def gated_norm_calls(dim, rows=64):
    lib = _lib.load()
    g = torch.Generator(device="cuda").manual_seed(dim)
    y, z = (torch.randn(rows, dim, generator=g, device="cuda") for _ in range(2))
    w, out = torch.randn(dim, generator=g, device="cuda"), torch.empty_like(y)

    def call(s):
        return lib.ssd_gated_rmsnorm(ptr(y), ptr(z), ptr(w), ptr(out), rows, dim, dim, 1e-5, _lib.SSD_F32,
                                     ctypes.c_void_p(s.cuda_stream))
    return [(call, [out])]


def chunk_out_calls(chunk, headdim):
    """The chunk output of f32 inputs, one head of two chunks."""
    import state_space_sequence_cumsum_gb300 as ssd
    lib, L, N = _lib.load(), 2 * chunk, 16
    g = torch.Generator(device="cuda").manual_seed(chunk + headdim)
    x = torch.randn(1, L, 1, headdim, generator=g, device="cuda")
    B, C = (torch.randn(1, L, 1, N, generator=g, device="cuda") for _ in range(2))
    dt, A, D = (torch.rand(s, generator=g, device="cuda") * m for s, m in (((1, L, 1), 0.1), ((1,), -1.0), ((1,), 1.0)))
    G, dt_t = ssd.ssd_chunk_cumsum(dt, A, chunk)
    states, _ = ssd.ssd_state_pass(x, B, dt_t, G, chunk)
    y = torch.empty_like(x)
    d = _lib.ssd_dims_t(1, L, 1, headdim, N, 1)

    def call(s):
        return lib.ssd_chunk_out(ptr(x), ptr(B), ptr(C), ptr(dt_t), ptr(G), ptr(states), ptr(D), ptr(y), d,
                                 _lib.SSD_F32, chunk, ctypes.c_void_p(s.cuda_stream))
    return [(call, [y])]


def test_gated_norms_and_chunk_outputs_of_two_sizes():
    # rows staged in 64 and 96 KB; chunk tiles of about 92 and 50 KB
    in_two_threads([gated_norm_calls(4096) + chunk_out_calls(256, 256),
                    gated_norm_calls(6144) + chunk_out_calls(128, 64)], rounds=200)
