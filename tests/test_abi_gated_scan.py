"""Host-side refusals of the gated scan and of the residual norm with dropout and in 8 bits
(CPU only: every case fails a check before anything is enqueued, so the fake addresses are
never read)."""
import math
import os

import pytest
import torch

from selective_state_space_ssd_amd import binding as bd
from test_abi_delta_norm import ALIAS, ALIGN, BIG, Call, DIM, GROUPS, NULL, OK, UNSUP, WS


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(bd.LIB_PATH):
        from selective_state_space_ssd_amd import build
        build.build()
    return bd.lib()


DIMS = dict(b=2, L=1000, D=256, sigmoid=0, io=1, a_io=0)
FWD = Call("ssd_gated_scan_fwd", ["x", "a", "init", "y", "states", "final", "ws"], dict(DIMS, ws_bytes=BIG),
           ["x", "a", "init", "y", "states", "final", "b", "L", "D", "sigmoid", "io", "a_io", "ws", "ws_bytes"])
BWD = Call("ssd_gated_scan_bwd", ["x", "a", "init", "states", "dy", "dfinal", "dx", "da", "dinit", "ws"], dict(DIMS, ws_bytes=BIG),
           ["x", "a", "init", "states", "dy", "dfinal", "dx", "da", "dinit", "b", "L", "D", "sigmoid", "io", "a_io", "ws", "ws_bytes"])
STEP = Call("ssd_gated_scan_step", ["state", "x", "a", "accept", "y", "out", "err"], dict(DIMS, L=4),
            ["state", "x", "a", "accept", "y", "out", "err", "b", "L", "D", "sigmoid", "io", "a_io"])
ROWS = dict(rows=10, D=256, eps=1e-5, p=0.1, io=1, res_io=0)
DROP = Call("ssd_norm_add_drop_fwd", ["x", "res", "scale", "w", "rng", "sum", "y"], ROWS,
            ["x", "res", "scale", "w", "rng", "sum", "y", "rows", "D", "eps", "p", "io", "res_io"])
DROP_B = Call("ssd_norm_add_drop_bwd", ["x", "sum", "scale", "w", "rng", "dy", "dsum", "dx", "dres", "dscale", "dw", "ws"], dict(ROWS, ws_bytes=BIG),
              ["x", "sum", "scale", "w", "rng", "dy", "dsum", "dx", "dres", "dscale", "dw", "rows", "D", "eps", "p", "io", "res_io", "ws", "ws_bytes"])
Q8 = Call("ssd_norm_add_q8_fwd", ["x", "res", "scale", "w", "sum", "q", "qs"], dict(rows=10, D=256, group=64, eps=1e-5, io=1, res_io=0),
          ["x", "res", "scale", "w", "sum", "q", "qs", "rows", "D", "group", "eps", "io", "res_io"])


@pytest.mark.parametrize("call,names", [
    (FWD, ["x", "a", "y"]), (BWD, ["x", "a", "dy", "dx", "da"]), (STEP, ["state", "x", "a", "y", "out"]),
    (DROP, ["x", "res", "w", "rng", "sum", "y"]), (DROP_B, ["x", "sum", "w", "rng", "dy", "dx", "dres", "dscale", "dw", "scale"]),
    (Q8, ["x", "res", "w", "sum", "q", "qs"])])
def test_null_pointers(lib, call, names):
    for n in names:
        assert call(lib, **{n: None}) == NULL, n


@pytest.mark.parametrize("call", [FWD, BWD, STEP])
@pytest.mark.parametrize("over,code", [
    (dict(b=-1), DIM), (dict(L=-1), DIM), (dict(D=0), DIM), (dict(D=-3), DIM), (dict(io=2), UNSUP), (dict(io=-1), UNSUP), (dict(a_io=2), UNSUP),
    (dict(io=0, a_io=1), UNSUP), (dict(b=65536), UNSUP), (dict(D=(1 << 31) - 256), UNSUP)])
def test_scan_dimensions(lib, call, over, code):
    assert call(lib, **over) == code


def test_scan_sizes_past_a_launch(lib):
    for call in (FWD, BWD):
        assert call(lib, b=65535, L=128 * 40, D=64) == UNSUP and call(lib, D=(1 << 24) + 1) == UNSUP
    assert STEP(lib, b=65535, D=64 * 40) == UNSUP


def test_scan_lengths(lib):
    for call in (FWD, BWD):
        assert call(lib, L=(1 << 31) - 64) == UNSUP
    for K in (0, 17, 100):
        assert STEP(lib, L=K) == UNSUP
    with pytest.raises(bd.SSDError):
        bd.ssd_gated_scan_fwd_workspace_bytes(1, 10, 0, 1, 1)
    with pytest.raises(bd.SSDError):
        bd.ssd_gated_scan_bwd_workspace_bytes(1, 10, 8, False, 0, 1)


@pytest.mark.parametrize("call,off", [
    (FWD, dict(x=8, a=4, init=4, y=2, states=8, final=8, ws=8)), (BWD, dict(x=8, a=4, init=4, states=8, dy=2, dfinal=8, dx=8, da=4, dinit=8, ws=8)),
    (STEP, dict(state=8, x=8, a=4, accept=2, y=2, out=8, err=1)), (DROP, dict(x=8, res=4, scale=8, w=4, rng=4, sum=8, y=2)),
    (DROP_B, dict(x=8, sum=4, scale=8, w=4, rng=4, dy=2, dsum=8, dx=8, dres=4, dscale=4, dw=8, ws=4)), (Q8, dict(x=8, res=4, scale=8, w=4, sum=8, q=8, qs=4))])
def test_alignment(lib, call, off):
    for n, o in off.items():
        assert call(lib, **{n: call.address(n, o)}) == ALIGN, n


@pytest.mark.parametrize("call,pairs", [
    (FWD, [("y", "x"), ("y", "a"), ("final", "init"), ("final", "y"), ("states", "x"), ("states", "y"), ("states", "final"), ("y", "init")]),
    (BWD, [("dx", "x"), ("dx", "dy"), ("da", "a"), ("da", "dx"), ("dinit", "dfinal"), ("dx", "states"), ("dinit", "da")]),
    (STEP, [("y", "x"), ("y", "state"), ("out", "a"), ("out", "y"), ("err", "accept"), ("err", "state"), ("err", "out")]),
    (DROP, [("sum", "x"), ("y", "x"), ("y", "res"), ("y", "sum"), ("sum", "rng"), ("y", "rng"), ("y", "scale")]),
    (DROP_B, [("dx", "x"), ("dx", "sum"), ("dres", "dsum"), ("dres", "dx"), ("dw", "dscale"), ("ws", "sum"), ("dx", "rng"), ("ws", "rng")]),
    (Q8, [("sum", "x"), ("q", "x"), ("q", "res"), ("q", "sum"), ("qs", "w"), ("qs", "q"), ("qs", "res"), ("qs", "sum")])])
def test_overlaps(lib, call, pairs):
    for out, other in pairs:
        assert call(lib, **{out: call.address(other)}) == ALIAS, (out, other)


def test_partial_overlaps(lib):
    assert STEP(lib, out=STEP.address("state", 1024)) == ALIAS
    assert DROP(lib, sum=DROP.address("res", 512)) == ALIAS and Q8(lib, sum=Q8.address("res", 512)) == ALIAS


def test_workspaces(lib):
    for with_states, states in ((True, BWD.address("states")), (False, None)):
        need = bd.ssd_gated_scan_bwd_workspace_bytes(2, 1000, 256, with_states, 1, 0)
        if need:
            assert BWD(lib, states=states, ws_bytes=need - 1) == WS and BWD(lib, states=states, ws=None) == WS
            assert BWD(lib, states=states, ws=BWD.address("dy")) == ALIAS and BWD(lib, states=states, ws=BWD.address("da")) == ALIAS
    # without states the workspace holds them
    more = need - bd.ssd_gated_scan_bwd_workspace_bytes(2, 1000, 256, True, 1, 0)
    assert more == 2 * 32 * 256 * 4
    need = bd.ssd_gated_scan_fwd_workspace_bytes(2, 1000, 256, 1, 0)
    if need:
        assert FWD(lib, ws_bytes=need - 1) == WS and FWD(lib, ws=None) == WS
        assert FWD(lib, ws=FWD.address("x")) == ALIAS and FWD(lib, ws=FWD.address("y")) == ALIAS
    need = bd.ssd_norm_bwd_workspace_bytes(10, 256, 256, 2, 1)
    assert DROP_B(lib, ws_bytes=need - 1) == WS and DROP_B(lib, ws=None) == WS


@pytest.mark.parametrize("p", [1.0, -0.1, 2.0, math.nan, math.inf])
def test_probabilities(lib, p):
    assert DROP(lib, p=p) == UNSUP and DROP_B(lib, p=p) == UNSUP


@pytest.mark.parametrize("over,code", [(dict(rows=-1), DIM), (dict(D=0), DIM), (dict(io=5), UNSUP), (dict(res_io=3), UNSUP), (dict(io=0, res_io=1), UNSUP)])
def test_norm_dimensions(lib, over, code):
    for call in (DROP, DROP_B, Q8):
        assert call(lib, **over) == code


def test_q8_groups(lib):
    assert Q8(lib, group=0) == DIM and Q8(lib, group=-8) == DIM and Q8(lib, group=96) == GROUPS and Q8(lib, group=512) == GROUPS
    assert Q8(lib, D=1 << 17, group=1) == UNSUP


def test_nothing_to_do(lib):
    assert STEP(lib, b=0) == OK and FWD(lib, b=0) == OK and BWD(lib, b=0) == OK
    assert FWD(lib, L=0, final=None) == OK and BWD(lib, L=0, dinit=None) == OK
    assert DROP(lib, rows=0) == OK and Q8(lib, rows=0) == OK


def test_binding_refuses_before_the_call():
    x, s = torch.zeros(2, 3, 8), torch.zeros(2, 8)
    with pytest.raises(ValueError):       # not on a GPU
        bd.gated_scan_step(s, x, x)
    with pytest.raises(ValueError):       # not [b, L, D]
        bd.gated_scan_fwd(s, s)
    with pytest.raises(ValueError):
        bd.norm_add_drop_fwd(s, s, torch.zeros(8), 1e-5, 0.1, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        bd.norm_add_q8_fwd(s, s, torch.zeros(8), 1e-5)
