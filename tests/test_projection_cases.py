"""The listed cases of perf/more_operators.py, and drawn ones, against that file's
64-bit definitions.

Tolerances (norm of the difference over the norm): half a step of the output's
type, bf16 2^-8; in f32 the rounding errors of the sums, 2e-5 as for the other
operators, which a plain f32 form stays within too.  8-bit values and their scales
are the definition's exactly in the quantiser; an optimiser's states are rounded
from f32 values, and one in some 10^5 may fall to the border's other side."""
import random

import pytest
import torch

from perf import more_operators as ops

pytestmark = pytest.mark.gpu

RNG = random.Random(11)
SMALL = [c for c in (ops.draw(RNG) for _ in range(120))
         if ops.work(c)["flops"] < 2e10 and ops.work(c)["bytes"] < 3e8][:24]
BOUND = {torch.bfloat16: 2.0 ** -8, torch.float32: 2e-5, torch.float8_e4m3fn: 1e-3}


def leaves(v):
    if isinstance(v, dict):
        return [x for k in sorted(v) for x in leaves(v[k])]
    return [x for t in v for x in leaves(t)] if isinstance(v, (tuple, list)) else [v]


@pytest.mark.parametrize("case", ops.listed() + SMALL, ids=lambda c: c.get("name") or "-".join(map(str, c.values())))
def test_case(case, monkeypatch):
    case = {k: v for k, v in case.items() if k != "name"}
    monkeypatch.setattr(ops, "own", True)
    got = leaves(ops.run(ops.prepare(case, 5)))
    want = ops.exact(case, 5)
    if want is None:  # too long in 64 bits: against the plain form
        monkeypatch.setattr(ops, "own", False)
        want = ops.run(ops.prepare(case, 5))
    want = leaves(want)
    assert len(got) == len(want)
    for a, b in zip(got, want):
        assert a.shape == b.shape
        if a.numel() == 0:
            continue
        a64, b64 = a.double(), b.double()
        assert bool(torch.isfinite(a64).all())
        bound = 0.0 if case["op"] == "quant" else BOUND[a.dtype]
        assert float((a64 - b64).norm()) <= bound * float(b64.norm())
