"""Limits of the gated delta rule's dimensions that the library checks before a launch (CPU
only: the addresses are never read)."""
import os

import pytest

from selective_state_space_ssd_amd import binding as bd

UNSUPPORTED, WORKSPACE, BASE, STEP = 4, 6, 0x7F0000000000, 1 << 44


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(bd.LIB_PATH):
        from selective_state_space_ssd_amd import build
        build.build()
    return bd.lib()


def calls(lib, L, P, N, io):
    p = [BASE + i * STEP for i in range(15)]
    dims = (1, L, 1, P, N, 1, 1.0, io)
    yield lib.ssd_gated_delta_fwd(*p[:8], *dims, None, 0, None)
    yield lib.ssd_gated_delta_bwd(*p[:14], *dims, None, 0, None)


@pytest.mark.parametrize("L", [(1 << 31) - 64, (1 << 31) - 1])
@pytest.mark.parametrize("P,N", [(16, 32), (20, 64), (64, 128)])
@pytest.mark.parametrize("io", [0, 1])
def test_tokens_past_the_counters(lib, L, P, N, io):
    assert all(st == UNSUPPORTED for st in calls(lib, L, P, N, io))
    with pytest.raises(bd.SSDError):
        bd.ssd_gated_delta_fwd_workspace_bytes(1, L, 1, P, N, 1, io)


@pytest.mark.parametrize("N,rows", [(16, 64), (32, 32), (256, 32)])
@pytest.mark.parametrize("io", [0, 1])
def test_state_rows_past_a_launch(lib, N, rows, io):
    p = [BASE + i * STEP for i in range(10)]
    for P in (((1 << 24) - 1) * rows + 1, (1 << 31) - 1):
        assert all(st == UNSUPPORTED for st in calls(lib, 2, P, N, io))
        assert lib.ssd_gated_delta_step(*p, 1, 1, 1, P, N, 1, 1.0, io, None) == UNSUPPORTED


def test_longest_that_is_counted(lib):
    """2^31 - 65 tokens are 2^25 - 1 chunks and a ragged one: a plan, and its workspace."""
    assert bd.ssd_gated_delta_fwd_workspace_bytes(1, (1 << 31) - 65, 1, 16, 32, 1, 1) > (1 << 31)
    assert next(calls(lib, (1 << 31) - 65, 16, 32, 1)) == WORKSPACE
