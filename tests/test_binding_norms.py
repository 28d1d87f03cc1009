"""What the norms' wrappers refuse before anything is enqueued (CPU only)."""
import os

import pytest
import torch

from selective_state_space_ssd_amd import binding as bd

BAD_DIM = 2


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(bd.LIB_PATH):
        from selective_state_space_ssd_amd import build
        build.build()


@pytest.mark.parametrize("rows", [0, 3])
def test_rows_of_no_channels(rows):
    """The gradients' wrappers ask for a workspace first: the library's refusal, not a division."""
    x, w = torch.zeros(rows, 0), torch.zeros(0)
    with pytest.raises(bd.SSDError) as e:
        bd.norm_gate_bwd(x, x, w, x, 1, 1e-5)
    assert e.value.status == BAD_DIM
    with pytest.raises(bd.SSDError) as e:
        bd.norm_add_bwd(x, x, w, x, None, 1e-5)
    assert e.value.status == BAD_DIM
