"""The gated scan's error word and limit of waits on the host's side (CPU only: every case fails a
check before anything is enqueued)."""
import os

import pytest
import torch

from selective_state_space_ssd_amd import binding as bd
from test_abi_delta_norm import ALIAS, ALIGN, BIG, Call, DIM, NULL, WS


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(bd.LIB_PATH):
        from selective_state_space_ssd_amd import build
        build.build()
    return bd.lib()


ERR = Call("ssd_gated_scan_workspace_error", ["ws", "err"], dict(ws_bytes=BIG, b=2, L=1000), ["ws", "ws_bytes", "b", "L", "err"])


def test_refusals(lib):
    assert ERR(lib, b=-1) == DIM and ERR(lib, L=-1) == DIM
    assert ERR(lib, err=None) == NULL and ERR(lib, L=100, err=None) == NULL
    assert ERR(lib, ws=ERR.address("ws", 8)) == ALIGN and ERR(lib, err=ERR.address("err", 2)) == ALIGN
    # a word only where blocks wait for each other
    assert ERR(lib, ws=None) == WS and ERR(lib, ws_bytes=15) == WS and ERR(lib, L=257, ws=None) == WS
    assert ERR(lib, ws_bytes=16, err=ERR.address("ws", 4)) == ALIAS and ERR(lib, L=256, err=ERR.address("ws", 4)) == ALIAS


def test_limit(lib):
    was = bd.ssd_gated_scan_wait_limit()
    assert was == 1 << 20
    try:
        assert bd.ssd_gated_scan_wait_limit(5) == was and bd.ssd_gated_scan_wait_limit(-1) == 5 and bd.ssd_gated_scan_wait_limit() == 5
        assert bd.ssd_gated_scan_wait_limit(0) == 5 and bd.ssd_gated_scan_wait_limit() == 0
    finally:
        bd.ssd_gated_scan_wait_limit(was)
    assert bd.ssd_gated_scan_wait_limit() == was


@pytest.mark.parametrize("L", [1, 128, 129, 255, 256, 257, 384, 512, 5000])
@pytest.mark.parametrize("b,D", [(1, 1), (2, 129), (64, 640), (300, 64), (1, 1 << 20)])
def test_which_calls_have_words(lib, L, b, D):
    """Sequences of more than 256 tokens use the workspace in both passes and for every type, and no
    shorter one does: that is where the error word is read."""
    for io in (0, 1):
        need = (bd.ssd_gated_scan_fwd_workspace_bytes(b, L, D, io, 0), bd.ssd_gated_scan_bwd_workspace_bytes(b, L, D, True, io, 0))
        assert all(n >= 16 for n in need) if L > 256 else need == (0, 0)


def test_binding_refuses_before_the_call():
    with pytest.raises(ValueError):         # not on a GPU
        bd.ssd_gated_scan_workspace_error(None, 1, 10, torch.zeros(1, dtype=torch.int32))
