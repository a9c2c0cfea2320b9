"""Refusals of the layer operators' Python calls (no GPU needed: they come
before the kernels are looked for)."""
import pytest
import torch

import state_space_sequence_cumsum_gb300 as ssd


@pytest.mark.parametrize("which", ["residual", "residual_out"])
@pytest.mark.parametrize("have,asked", [(torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)])
def test_a_residual_of_another_type_than_the_one_asked_for(which, have, asked):
    y, w = torch.zeros(2, 8, dtype=torch.bfloat16), torch.ones(8)
    given = {"residual": None, which: torch.zeros(2, 8, dtype=have)}
    with pytest.raises(TypeError, match=f"{which} is {have}, residual_dtype {asked}"):
        ssd.ssd_block_norm(y, weight=w, residual_dtype=asked, **given)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_residual_of_the_type_asked_for_passes_this_check(dtype):
    y, w = torch.zeros(2, 8, dtype=torch.bfloat16), torch.ones(8)
    with pytest.raises(ValueError, match="CUDA tensors"):
        ssd.ssd_block_norm(y, torch.zeros(2, 8, dtype=dtype), w, residual_dtype=dtype)
