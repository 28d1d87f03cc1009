"""Counts of accepted tokens out of range, seen by a caller of the allocating wrapper (MI355X
only)."""
import pytest
import torch

from delta_helpers import inputs_of, make
from selective_state_space_ssd_amd import binding as bd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("counts,flagged", [([4, 0, 2], 0), ([4, 5, 2], 1), ([-1, 0, 4], 1)])
def test_error_flag(counts, flagged):
    c = make(3, 4, 2, 1, 32, 64, torch.bfloat16, seed=1)
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    acc = torch.tensor(counts, dtype=torch.int32, device="cuda")
    y, S = bd.gated_delta_step(c["init_state"], *inputs_of(c), 0.5, accept_len=acc, err_flag=flag)
    y2, S2 = bd.gated_delta_step(c["init_state"], *inputs_of(c), 0.5, accept_len=acc.clamp(0, 4))
    assert int(flag) == flagged and torch.equal(y, y2) and torch.equal(S, S2)
