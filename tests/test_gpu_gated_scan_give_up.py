"""Waits of the gated scan that give up: they end, leave NaN in what depends on them and nothing
else, and say so in the workspace (MI355X only).  A limit of no looks makes every wait give up
from the host's side: the kernels run and end as always."""
import pytest
import torch

from scan_helpers import make
from selective_state_space_ssd_amd import binding as bd

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
TILE = 256      # no block holds more tokens, and none of several fewer than 128

# b, L, D: few short blocks, many of long tiles, a chain of more blocks than are looked back over,
# one and two channels a lane
SHAPES = [(2, 700, 96), (1, 1025, 33), (4, 700, 2050), (1, 30000, 34), (2, 9217, 1)]


@pytest.fixture
def limit():
    was = bd.ssd_gated_scan_wait_limit()
    yield bd.ssd_gated_scan_wait_limit
    bd.ssd_gated_scan_wait_limit(was)


def workspace(b, L, D, dtype):
    io = bd.SSD_DTYPE_BF16 if dtype == BF else bd.SSD_DTYPE_F32
    n = max(16, bd.ssd_gated_scan_fwd_workspace_bytes(b, L, D, io, bd.SSD_DTYPE_F32), bd.ssd_gated_scan_bwd_workspace_bytes(b, L, D, False, io, bd.SSD_DTYPE_F32))
    return torch.full((n,), 255, dtype=torch.uint8, device="cuda")


def error(ws, b, L):
    flag = torch.full((1,), 77, dtype=torch.int32, device="cuda")
    bd.ssd_gated_scan_workspace_error(ws, b, L, flag)
    return int(flag)


@pytest.mark.parametrize("b,L,D", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_a_wait_that_gives_up(b, L, D, dtype, sigmoid, limit):
    c = make(b, L, D, sigmoid, dtype, F32, seed=L)
    ws = workspace(b, L, D, dtype)

    def fwd():
        return bd.gated_scan_fwd(c["x"], c["a"], sigmoid=sigmoid, init_state=c["init"], keep_states=True, workspace=ws)

    def bwd(states):
        return bd.gated_scan_bwd(c["x"], c["a"], c["dy"], sigmoid=sigmoid, init_state=c["init"], d_final=c["d_final"], states=states, workspace=ws)

    good = fwd()
    assert error(ws, b, L) == 0
    kept = good[2]
    grads = bwd(kept)
    assert error(ws, b, L) == 0
    limit(0)
    y, final, states = fwd()
    assert error(ws, b, L) == 1
    assert torch.equal(y[:, :128], good[0][:, :128]) and bool(y[:, TILE:].isnan().all()) and bool(final.isnan().all())
    assert torch.equal(states[:, :4], kept[:, :4]) and bool(states[:, TILE // 32 + 1:].isnan().all())
    dx, da, d_init = bwd(kept)
    assert error(ws, b, L) == 1
    last = (L - 1) // 128 * 128         # in the last block, whatever its size
    assert torch.equal(dx[:, last:], grads[0][:, last:]) and torch.equal(da[:, last:], grads[1][:, last:])
    assert all(bool(t[:, :L - TILE].isnan().all()) for t in (dx, da)) and bool(d_init.isnan().all())
    bwd(None)
    assert error(ws, b, L) == 1
    # and the same workspace serves the next calls
    limit(1 << 20)
    assert all(torch.equal(s, t) for s, t in zip(fwd(), good)) and error(ws, b, L) == 0
    assert all(torch.equal(s, t) for s, t in zip(bwd(kept), grads)) and error(ws, b, L) == 0
    bwd(None)
    assert error(ws, b, L) == 0


@pytest.mark.parametrize("L", [0, 1, 128, 129, 256])
@pytest.mark.parametrize("b,D", [(1, 64), (64, 640)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_sequences_of_one_block_wait_for_nothing(b, L, D, dtype, limit):
    c = make(b, L, D, True, dtype, F32, seed=L)
    ws = workspace(b, L, D, dtype)
    run = lambda: bd.gated_scan_fwd(c["x"], c["a"], sigmoid=True, init_state=c["init"], workspace=ws) + bd.gated_scan_bwd(
        c["x"], c["a"], c["dy"], sigmoid=True, init_state=c["init"], d_final=c["d_final"], workspace=ws)
    want = run()
    limit(0)
    assert all(torch.equal(s, t) for s, t in zip(run(), want))
    assert error(ws, b, L) == 0 and error(None, b, L) == 0 and error(ws, 0, 5000) == 0


def test_a_captured_call_keeps_its_limit(limit):
    c = make(1, 3000, 64, True, BF, F32, seed=1)
    ws, y = workspace(1, 3000, 64, BF), torch.empty_like(c["x"])
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = bd.gated_scan_fwd(c["x"], c["a"], sigmoid=True)[0]

    def step():
        bd.ssd_gated_scan_fwd(c["x"], c["a"], None, y, None, None, True, ws)
        bd.ssd_gated_scan_workspace_error(ws, 1, 3000, flag)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    limit(0)
    for _ in range(3):
        y.zero_()
        flag.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and int(flag) == 0
        step()
        torch.cuda.synchronize()
        assert bool(y[:, TILE:].isnan().all()) and int(flag) == 1
