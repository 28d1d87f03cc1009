"""Host-side refusals of the gated delta rule and of the norms (CPU only: every case fails
a check before anything is enqueued, so the fake addresses are never read)."""
import os

import pytest
import torch

from selective_state_space_ssd_amd import binding as bd

OK, NULL, DIM, GROUPS, UNSUP, ALIGN, WS, ALIAS, HIP = range(9)
BASE = 0x7F0000000000
STEP = 0x100000000
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(bd.LIB_PATH):
        from selective_state_space_ssd_amd import build
        build.build()
    return bd.lib()


class Call:
    """A C call by argument names, with valid fake arguments to start from."""

    def __init__(self, name, pointers, values, order):
        self.name, self.pointers, self.values, self.order = name, pointers, values, order

    def address(self, pointer, off=0):
        return BASE + self.pointers.index(pointer) * STEP + off

    def __call__(self, lib, **over):
        args = {p: self.address(p) for p in self.pointers}
        args.update(self.values)
        args.update(over)
        return getattr(lib, self.name)(*[args[n] for n in self.order], None)


DIMS = dict(b=2, L=100, H=4, P=64, N=64, G=2, scale=1.0, io=1)
FWD = Call("ssd_gated_delta_fwd", ["q", "k", "v", "a", "beta", "init", "y", "final", "ws"], dict(DIMS, ws_bytes=BIG),
           ["q", "k", "v", "a", "beta", "init", "y", "final", "b", "L", "H", "P", "N", "G", "scale", "io", "ws", "ws_bytes"])
STEPC = Call("ssd_gated_delta_step", ["state", "q", "k", "v", "a", "beta", "accept", "y", "out", "err"], dict(DIMS, L=4),
             ["state", "q", "k", "v", "a", "beta", "accept", "y", "out", "err", "b", "L", "H", "P", "N", "G", "scale", "io"])
BWD = Call("ssd_gated_delta_bwd", ["q", "k", "v", "a", "beta", "init", "dy", "dfinal", "dq", "dk", "dv", "da", "dbeta", "dinit", "ws"],
           dict(DIMS, ws_bytes=BIG), ["q", "k", "v", "a", "beta", "init", "dy", "dfinal", "dq", "dk", "dv", "da", "dbeta", "dinit",
                                      "b", "L", "H", "P", "N", "G", "scale", "io", "ws", "ws_bytes"])
ROWS = dict(rows=10, D=256, group=64, eps=1e-5, gate_first=0, io=1)
GATE = Call("ssd_norm_gate_fwd", ["x", "z", "w", "y"], ROWS, ["x", "z", "w", "y", "rows", "D", "group", "eps", "gate_first", "io"])
GATE_B = Call("ssd_norm_gate_bwd", ["x", "z", "w", "dy", "dx", "dz", "dw", "ws"], dict(ROWS, ws_bytes=BIG),
              ["x", "z", "w", "dy", "dx", "dz", "dw", "rows", "D", "group", "eps", "gate_first", "io", "ws", "ws_bytes"])
ADD = Call("ssd_norm_add_fwd", ["x", "res", "scale", "w", "sum", "y"], dict(rows=10, D=256, eps=1e-5, io=1, res_io=0),
           ["x", "res", "scale", "w", "sum", "y", "rows", "D", "eps", "io", "res_io"])
ADD_B = Call("ssd_norm_add_bwd", ["x", "sum", "scale", "w", "dy", "dsum", "dx", "dres", "dscale", "dw", "ws"],
             dict(rows=10, D=256, eps=1e-5, io=1, res_io=0, ws_bytes=BIG),
             ["x", "sum", "scale", "w", "dy", "dsum", "dx", "dres", "dscale", "dw", "rows", "D", "eps", "io", "res_io", "ws", "ws_bytes"])


@pytest.mark.parametrize("call,names", [
    (FWD, ["q", "k", "v", "a", "beta", "y"]), (STEPC, ["state", "q", "k", "v", "a", "beta", "y", "out"]),
    (BWD, ["q", "k", "v", "a", "beta", "dy", "dq", "dk", "dv", "da", "dbeta"]),
    (GATE, ["x", "w", "y"]), (GATE_B, ["x", "z", "w", "dy", "dx", "dz", "dw"]), (ADD, ["x", "res", "w", "sum", "y"]),
    (ADD_B, ["x", "sum", "scale", "w", "dy", "dx", "dres", "dscale", "dw"])])
def test_null_pointers(lib, call, names):
    for n in names:
        assert call(lib, **{n: None}) == NULL, n


@pytest.mark.parametrize("call", [FWD, STEPC, BWD])
@pytest.mark.parametrize("over,code", [
    (dict(b=-1), DIM), (dict(L=-1), DIM), (dict(H=0), DIM), (dict(P=0), DIM), (dict(N=0), DIM), (dict(G=0), DIM), (dict(G=-2), DIM),
    (dict(G=3), GROUPS), (dict(N=24), UNSUP), (dict(N=48), UNSUP), (dict(N=512), UNSUP), (dict(io=2), UNSUP), (dict(io=-1), UNSUP),
    (dict(b=65536), UNSUP), (dict(H=65536), UNSUP)])
def test_delta_dimensions(lib, call, over, code):
    assert call(lib, **over) == code


@pytest.mark.parametrize("over", [dict(P=24), dict(P=1), dict(N=16), dict(N=256, io=0), dict(H=65534, G=65534, P=256)])
def test_backward_shapes(lib, over):
    assert BWD(lib, **over) == UNSUP


@pytest.mark.parametrize("K", [0, 17, 100])
def test_step_token_counts(lib, K):
    assert STEPC(lib, L=K) == UNSUP


@pytest.mark.parametrize("call,off", [
    (FWD, dict(q=8, k=2, v=8, y=4, init=8, final=4, a=2, beta=1, ws=8)),
    (STEPC, dict(state=8, out=8, q=8, k=4, v=1, y=1, a=2, beta=2, accept=2, err=1)),
    (BWD, dict(q=8, k=4, v=2, a=2, beta=1, init=8, dy=8, dfinal=4, dq=8, dk=2, dv=4, da=2, dbeta=2, dinit=8, ws=8)),
    (GATE, dict(x=8, z=2, w=4, y=8)), (GATE_B, dict(x=8, z=2, w=4, dy=8, dx=4, dz=2, dw=8, ws=8)),
    (ADD, dict(x=8, res=4, scale=4, w=8, sum=8, y=2)),
    (ADD_B, dict(x=8, sum=4, scale=8, w=4, dy=2, dsum=8, dx=8, dres=4, dscale=4, dw=8, ws=4))])
def test_alignment(lib, call, off):
    for n, o in off.items():
        assert call(lib, **{n: call.address(n, o)}) == ALIGN, n


@pytest.mark.parametrize("call,pairs", [
    (FWD, [("y", "q"), ("y", "v"), ("y", "a"), ("final", "init"), ("final", "k"), ("final", "y"), ("y", "init")]),
    (STEPC, [("y", "v"), ("out", "q"), ("y", "state"), ("out", "y"), ("err", "accept"), ("err", "state"), ("out", "beta")]),
    (BWD, [("dq", "q"), ("dk", "dq"), ("dv", "v"), ("dv", "dy"), ("da", "a"), ("dbeta", "da"), ("dinit", "dfinal"), ("dinit", "init"), ("ws", "k"), ("ws", "dv")]),
    (GATE, [("y", "x"), ("y", "z"), ("y", "w")]), (GATE_B, [("dx", "x"), ("dz", "dx"), ("dw", "w"), ("ws", "dy"), ("ws", "dx"), ("dx", "dy")]),
    (ADD, [("sum", "x"), ("y", "x"), ("y", "res"), ("y", "sum"), ("sum", "w"), ("y", "scale")]),
    (ADD_B, [("dx", "x"), ("dx", "sum"), ("dres", "dsum"), ("dres", "dx"), ("dw", "dscale"), ("ws", "sum"), ("dscale", "scale")])])
def test_overlaps(lib, call, pairs):
    for out, other in pairs:
        assert call(lib, **{out: call.address(other)}) == ALIAS, (out, other)


def test_partial_overlaps(lib):
    assert STEPC(lib, out=STEPC.address("state", 1024)) == ALIAS
    assert ADD(lib, sum=ADD.address("res", 512)) == ALIAS


@pytest.mark.parametrize("call", [GATE, GATE_B])
@pytest.mark.parametrize("over,code", [(dict(rows=-1), DIM), (dict(D=0), DIM), (dict(group=0), DIM), (dict(group=96), GROUPS), (dict(io=5), UNSUP),
                                       (dict(rows=1 << 30, D=64, group=1), UNSUP), (dict(D=1 << 17, group=1), UNSUP)])
def test_norm_gate_dimensions(lib, call, over, code):
    assert call(lib, **over) == code


@pytest.mark.parametrize("call", [ADD, ADD_B])
@pytest.mark.parametrize("over,code", [(dict(rows=-1), DIM), (dict(D=0), DIM), (dict(io=5), UNSUP), (dict(res_io=3), UNSUP), (dict(io=0, res_io=1), UNSUP)])
def test_norm_add_dimensions(lib, call, over, code):
    assert call(lib, **over) == code


@pytest.mark.parametrize("call", [GATE_B, ADD_B])
def test_norm_workspace(lib, call):
    assert call(lib, ws=None) == WS
    need = bd.ssd_norm_bwd_workspace_bytes(10, 256, 64 if call is GATE_B else 256, 1 if call is GATE_B else 2, 1)
    assert need > 0 and call(lib, ws_bytes=need - 1) == WS


def test_delta_workspace(lib):
    assert FWD(lib, ws=None) == WS
    need = bd.ssd_gated_delta_fwd_workspace_bytes(2, 100, 4, 64, 64, 2, 1)
    assert need > 0 and FWD(lib, ws_bytes=need - 1) == WS
    for name in ("q", "v", "y", "final"):
        assert FWD(lib, ws=FWD.address(name)) == ALIAS
    assert BWD(lib, ws=None) == WS
    need = bd.ssd_gated_delta_bwd_workspace_bytes(2, 100, 4, 64, 64, 2, 1)
    assert need > 0 and BWD(lib, ws_bytes=need - 1) == WS


def test_workspace_sizes():
    with pytest.raises(bd.SSDError):
        bd.ssd_gated_delta_fwd_workspace_bytes(1, 10, 4, 64, 40, 2, 1)
    with pytest.raises(bd.SSDError):
        bd.ssd_norm_bwd_workspace_bytes(10, 256, 100, 1, 1)
    with pytest.raises(bd.SSDError):
        bd.ssd_norm_bwd_workspace_bytes(10, 256, 64, 3, 1)
    assert bd.ssd_norm_bwd_workspace_bytes(0, 256, 64, 1, 1) == 0


def test_nothing_to_do(lib):
    assert STEPC(lib, b=0) == OK and FWD(lib, b=0) == OK and BWD(lib, b=0) == OK
    assert FWD(lib, L=0, final=None) == OK and BWD(lib, L=0, dinit=None) == OK
    assert GATE(lib, rows=0) == OK and ADD(lib, rows=0) == OK


def test_binding_refuses_before_the_call():
    t = torch.zeros(2, 3, 4, 8)
    g = torch.zeros(2, 3, 4)
    with pytest.raises(ValueError):       # not on a GPU
        bd.gated_delta_step(torch.zeros(2, 4, 8, 8), t, t, t, g, g, 1.0)
    with pytest.raises(ValueError):
        bd.norm_gate_fwd(torch.zeros(2, 8), None, torch.zeros(8), 8, 1e-5)
