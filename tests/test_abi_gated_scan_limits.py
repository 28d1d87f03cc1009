"""The gated scan's sizes on both sides of their limits, through the workspace queries and refused
calls (CPU only: nothing is enqueued)."""
import os

import pytest

from selective_state_space_ssd_amd import binding as bd
from test_abi_delta_norm import NULL, OK, UNSUP
from test_abi_gated_scan import BWD, FWD, STEP


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(bd.LIB_PATH):
        from selective_state_space_ssd_amd import build
        build.build()
    return bd.lib()


TILES = 1 << 21     # b ceil(L / 128) ceil(D / 64)
WITHIN = [(1, 1 << 28, 1), (1, 1 << 28, 64), (2, 1 << 27, 64), (1, 1024, 1 << 24), (65535, 32 * 128, 64), (32768, 128, 4096)]
BEYOND = [(1, (1 << 28) + 1, 1), (1, (1 << 28) + 1, 64), (1, 1 << 28, 65), (3, 1 << 27, 64), (1, 1025, 1 << 24), (1, 128, (1 << 24) + 1), (65535, 33 * 128, 64),
          (32768, 129, 4096), (1, (1 << 31) - 1, 1)]


def tiles(b, L, D):
    return b * -(-L // 128) * -(-D // 64)


@pytest.mark.parametrize("io,a_io", [(0, 0), (1, 0), (1, 1)])
def test_workspaces_on_both_sides(lib, io, a_io):
    for b, L, D in WITHIN:
        assert tiles(b, L, D) <= TILES
        fwd = bd.ssd_gated_scan_fwd_workspace_bytes(b, L, D, io, a_io)
        bwd = bd.ssd_gated_scan_bwd_workspace_bytes(b, L, D, True, io, a_io)
        # a word of 8 bytes for every channel of a block, blocks of at least 128 tokens
        assert all(n <= 16 + 8 * 128 * tiles(b, L, D) + 16 for n in (fwd, bwd))
        assert bd.ssd_gated_scan_bwd_workspace_bytes(b, L, D, False, io, a_io) == bwd + b * -(-L // 32) * D * 4
    for b, L, D in BEYOND:
        assert tiles(b, L, D) > TILES or D > 1 << 24
        for query in (lambda: bd.ssd_gated_scan_fwd_workspace_bytes(b, L, D, io, a_io), lambda: bd.ssd_gated_scan_bwd_workspace_bytes(b, L, D, True, io, a_io)):
            with pytest.raises(bd.SSDError):
                query()


def test_calls_on_both_sides(lib):
    # within: the next check refuses (a missing output), beyond: the sizes do
    for b, L, D in WITHIN:
        assert FWD(lib, b=b, L=L, D=D, y=None) == NULL and BWD(lib, b=b, L=L, D=D, dx=None) == NULL
    for b, L, D in BEYOND:
        assert FWD(lib, b=b, L=L, D=D, y=None) == UNSUP and BWD(lib, b=b, L=L, D=D, dx=None) == UNSUP
    assert STEP(lib, b=32768, L=16, D=4096, y=None) == NULL and STEP(lib, b=32768, L=1, D=4097, y=None) == UNSUP
    assert STEP(lib, b=1, L=1, D=1 << 24, y=None) == NULL and STEP(lib, b=1, L=1, D=(1 << 24) + 1, y=None) == UNSUP


def test_no_sequences_are_nothing_to_do_at_any_length(lib):
    for L in (0, 1 << 28, 1 << 30, (1 << 31) - 1):
        assert FWD(lib, b=0, L=L) == OK and BWD(lib, b=0, L=L) == OK
