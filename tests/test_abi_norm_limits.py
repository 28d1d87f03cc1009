"""Limits of the norms' dimensions that the library checks before a launch (CPU only: the
addresses are never read)."""
import os

import pytest

from selective_state_space_ssd_amd import binding as bd

UNSUPPORTED, BASE, STEP = 4, 0x7F0000000000, 1 << 40


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(bd.LIB_PATH):
        from selective_state_space_ssd_amd import build
        build.build()
    return bd.lib()


@pytest.mark.parametrize("D", [(1 << 31) - 256, (1 << 31) - 64, (1 << 31) - 1])
@pytest.mark.parametrize("io", [0, 1])
def test_channels_past_the_counters(lib, D, io):
    """Channel counters of 32 bits run up to a block past the last channel: beyond 2^31 they
    would be negative."""
    p = [BASE + i * STEP for i in range(11)]
    assert lib.ssd_norm_gate_fwd(p[0], p[1], p[2], p[3], 1, D, D, 1e-5, 0, io, None) == UNSUPPORTED
    assert lib.ssd_norm_gate_bwd(*p[:7], 1, D, D, 1e-5, 0, io, p[7], 1 << 62, None) == UNSUPPORTED
    assert lib.ssd_norm_add_fwd(*p[:6], 1, D, 1e-5, io, io, None) == UNSUPPORTED
    assert lib.ssd_norm_add_bwd(*p[:10], 1, D, 1e-5, io, io, p[10], 1 << 62, None) == UNSUPPORTED
    with pytest.raises(bd.SSDError):
        bd.ssd_norm_bwd_workspace_bytes(1, D, D, 1, io)
