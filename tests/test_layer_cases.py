"""The layer operators on sizes that take their long paths -- runs of many
groups of tokens, blocks that walk several chunks, rows and items -- and on the
listed cases of perf/operators.py, against that file's 64-bit definitions.

Tolerances.  Element by element those of test_layer.py, for its reasons.  The
scan's bound of 600 decays holds here too: steps average 1e-3 and more and rates
are 1 and more, and a contribution's s decays weigh at most
max s e^(-s/1000) = 368.
As a whole (norm of the difference over the norm), a kernel may be off by what
the plain f32 form is, and by its fast exponentials and reciprocals: 2^-21, and
in a scan sqrt(368) 2^-22 for the decays of one recurrence, as errors of their
own, twice that with the reverse one."""
import math

import pytest
import torch

from perf import operators as ops
from state_space_sequence_cumsum_gb300 import _lib

PLAIN, SCAN = 2e-5, 1.5e-4
SMS = 152  # also what the sizes are planned for where there is no device

CONVS = [  # a run of 24 tokens or more; lengths that are no multiple of it or of a group of four
    ops.conv_case("conv_grad", 4, 1501, 4096, 4, "bf16", carry=True, row=4160, name="bf16_vectors"),
    ops.conv_case("conv_grad", 4, 1503, 2048, 3, "f32", name="f32_vectors"),
    ops.conv_case("conv_grad", 4, 1498, 2701, 4, "bf16", carry=True, row=2707, name="bf16_a_warp_apart"),
    ops.conv_case("conv_grad", 4, 1501, 1537, 2, "f32", carry=True, row=1541, name="f32_single"),
    ops.conv_case("conv_grad", 8, 10667, 33, 4, "bf16", carry=True, name="bf16_single"),
]
SCANS = [  # three chunks a block of the gradients or more, the last one short
    ops.scan_case("scan_grad", 2, 1021, 3840, 16, 1, "bf16", carry=True, row=7680, name="states16_bf16"),
    ops.scan_case("scan_grad", 2, 1021, 3837, 16, 1, "f32", gated=False, row=3841, name="states16_f32_odd"),
    ops.scan_case("scan_grad", 2, 701, 960, 64, 1, "f32", carry=True, name="states64_f32"),
    ops.scan_case("scan_grad", 2, 1021, 1920, 32, 1, "bf16", carry=True, name="states32_bf16"),
    ops.scan_case("scan_grad", 2, 1021, 7680, 8, 2, "bf16", name="states8_bf16_groups"),
    ops.scan_case("scan_grad", 4, 1021, 7679, 3, 1, "bf16", carry=True, name="states3_bf16_odd"),
]
NORMS = [  # several rows an item, or several items a block
    ops.norm_case("norm_grad", 1001, 2560, "bf16", "f32", gate_rows=1001, name="a_gate_row_per_token"),
    ops.norm_case("norm_grad", 6000, 2560, "bf16", "f32", name="twenty_rows_an_item"),
    ops.norm_case("norm_grad", 6002, 2560, "f32", "f32", gate_rows=2, name="f32_two_gate_rows"),
    ops.norm_case("norm_grad", 3000, 1001, "f32", "f32", gate_rows=500, name="odd_width_six_rows_a_gate"),
    ops.norm_case("norm_grad", 2500, 6400, "bf16", "f32", name="wide_four_rows"),
    ops.norm_case("norm_grad", 1300, 6400, "bf16", "bf16", gate_rows=1300, name="wide_two_items_a_block"),
    ops.norm_case("norm_grad", 2000, 2303, "bf16", "f32", gate_rows=2, post=False, name="wide_odd"),
]


def ceil(a, b):
    return -(-a // b)


def up256(n):
    return ceil(n, 256) * 256


# ------------------------------------------------- the plans of these sizes

def pick_run(seqlen, slots, start, blocks):
    best, least = 4, None
    for run in range(4, 257, 4):
        waves = ceil(blocks(run), slots)
        if least is None or waves * (run + start) < least:
            best, least = run, waves * (run + start)
        if waves == 1 or run >= seqlen:
            break
    return best


@pytest.mark.parametrize("case", CONVS, ids=lambda c: c["name"])
def test_convolutions_walk_long_runs(case):
    b, L, D, W = (case[k] for k in ("batch", "seqlen", "dim", "width"))
    size = _lib.load().ssd_causal_conv_bwd_workspace_size(_lib.ssd_conv_dims_t(b, L, D, W))
    parts = size // (4 * (W + 1) * D * b)  # of a sequence, four runs each, in the layout that has the most
    assert parts >= 1 and L / (4 * parts) >= 24
    for columns in (D // 4, ceil(D, 64) * 32, D):
        if (columns == D // 4) == (D % 4 == 0):
            assert pick_run(L, SMS * 3, 8, lambda r: ceil(b * columns * ceil(L, r), 256)) >= 24


def scan_plan(case):
    """(chunks a block of the gradients, the backward's workspace with given chunk states)"""
    b, L, D, N, G = (case[k] for k in ("batch", "seqlen", "dim", "dstate", "ngroups"))
    nc, kpg = ceil(L, 16), D // G
    lanes = 1
    while 4 * lanes < N:
        lanes *= 2
    reverse = 0
    for held in ({1: 3, 2: 5, 4: 9, 8: 4, 16: 2}[lanes], {1: 3, 2: 5, 4: 8, 8: 4, 16: 2}[lanes]):
        cb = {1: 64, 2: 32}.get(lanes, 16)
        n = min(held * SMS // (G * ceil(kpg, cb) * b), nc // 4)
        if n > 1:
            segments = ceil(nc, ceil(nc, n))
            reverse = max(reverse, 4 * b * (segments * D * (N + 1) + nc * D))
    nblk = ceil(kpg, 256 // lanes)
    cols = nblk * G * b
    n = max(1, min(nc, max(min(SMS * 40 // cols, nc // 4), SMS * 12 // cols)))
    chunks = ceil(nc, n)
    items = b * ceil(nc, chunks)
    grad = 2 * up256(4 * G * nblk * b * L * N) + up256(4 * items * D * N) + up256(8 * items * D)
    return chunks, up256(4 * b * nc * D * N) + up256(reverse) + grad


@pytest.mark.parametrize("case", SCANS, ids=lambda c: c["name"])
def test_scan_gradients_walk_several_chunks(case):
    chunks, size = scan_plan(case)
    assert chunks >= 3
    dims = _lib.ssd_scan_dims_t(*[case[k] for k in ("batch", "seqlen", "dim", "dstate", "ngroups")])
    assert _lib.load().ssd_selective_scan_bwd_workspace_size(dims, 1) == size  # the plan above is the library's


def norm_plan(case):
    """(items, blocks that walk them, rows an item at least, the backward's workspace)"""
    T, D, rows = case["tokens"], case["dim"], case["gate_rows"]
    vectors = D // 4 if D % 4 == 0 else D
    teams = [ceil(vectors, 32 * v) * 32 for v in (1, 2, 4)]
    team = next((t for t in teams if t <= 320), None)
    held = 4 if team is None else 16 if team <= 48 else 2 if team > 256 else 768 // team
    groups = max(rows, 1)
    per = T // groups
    spans = min(ceil(SMS * held, groups), per // (1 if per < 128 else 2 if per < 256 else 4))
    blocks = min(groups * spans, SMS * held)
    lines = 2 * blocks + (groups * spans if rows and spans > 1 else 0)
    return groups * spans, blocks, per // spans, up256(4 * lines * D)


@pytest.mark.parametrize("case", NORMS, ids=lambda c: c["name"])
def test_norm_gradients_walk_several_rows_or_items(case):
    items, blocks, rows, size = norm_plan(case)
    assert rows >= 4 or items > blocks
    assert _lib.load().ssd_block_norm_bwd_workspace_size(case["tokens"], case["dim"], case["gate_rows"]) == size


# ----------------------------------------------------------------- the results

def pairs(got, want):
    if isinstance(want, dict):
        assert set(got) == set(want)
        got, want = [got[k] for k in want], list(want.values())
    for g, w in zip(got, want, strict=True):
        assert (g is None) == (w is None)
        if w is not None:
            yield g, w


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


def check(case, seed):
    want = ops.exact(case, seed)
    assert want is not None
    state = ops.prepare(case, seed)
    ops.own = True
    try:
        got = ops.run(state)
    finally:
        ops.own = False
    plain = ops.run(state)
    scan, grad = case["op"].startswith("scan"), case["op"] == "scan_grad"
    tol = SCAN * (2 if grad else 1) if scan else PLAIN
    more = math.sqrt(368) * 2.0 ** -22 * (2 if grad else 1) if scan else 2.0 ** -21
    for (g, w), (p, _) in zip(pairs(got, want), pairs(plain, want)):
        assert g.shape == w.shape and bool(torch.isfinite(g).all())
        w = w.double()
        bound = tol * (w.abs() + w.square().mean().sqrt())
        if g.dtype == torch.bfloat16:
            bound += 2.0 ** -8 * w.abs()
        assert bool(((g.double() - w).abs() <= bound).all())
        assert off(g, w) <= off(p, w) + more


@pytest.mark.gpu
@pytest.mark.parametrize("case", CONVS + SCANS + NORMS, ids=lambda c: c["name"])
def test_long_paths(case):
    assert torch.cuda.get_device_properties(0).multi_processor_count == SMS
    forward = dict(case, op=case["op"].removesuffix("_grad"))
    check(case, 5)
    if case["op"] != "scan_grad":  # which returns the forward's results too
        check(forward, 6)


@pytest.mark.gpu
@pytest.mark.parametrize("case", ops.listed(), ids=lambda c: c["name"])
def test_listed_cases(case):
    check(case, 7)
    torch.cuda.empty_cache()
