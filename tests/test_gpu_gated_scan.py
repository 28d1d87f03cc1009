"""The gated scan against its float64 form, token by token (MI355X only).  Tolerances:
scan_helpers.tol."""
import math

import pytest
import torch

from oracle import gated_scan as oracle
from scan_helpers import U, check_bwd, check_fwd, make, rel, tol
from selective_state_space_ssd_amd import binding as bd

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
TYPES = [(BF, BF), (BF, F32), (F32, F32)]

# b, L, D: one token, the last token of a kept state's stretch and one beyond, single and odd
# channels, channels next to a strip of lanes, one tile of tokens and next to it, many tiles
SHAPES = [(1, 1, 1), (2, 1, 130), (1, 31, 7), (3, 32, 64), (1, 33, 65), (2, 77, 512), (1, 127, 129), (1, 128, 128), (2, 129, 127),
          (1, 255, 66), (1, 256, 2), (2, 257, 62), (1, 512, 256), (1, 513, 254), (2, 700, 96), (3, 1025, 33), (1, 3000, 130), (1, 5000, 3), (5, 2047, 64)]


def run_bwd(c, sigmoid, states=None, d_final=True):
    return bd.gated_scan_bwd(c["x"], c["a"], c["dy"], sigmoid=sigmoid, init_state=c["init"], d_final=c["d_final"] if d_final else None, states=states)


@pytest.mark.parametrize("b,L,D", SHAPES)
@pytest.mark.parametrize("dtype,a_dtype", TYPES)
@pytest.mark.parametrize("sigmoid", [False, True])
def test_forward_and_gradients(b, L, D, dtype, a_dtype, sigmoid):
    c = make(b, L, D, sigmoid, dtype, a_dtype, seed=L + D, init=(L + D) % 3 != 0)
    y, final, kept = bd.gated_scan_fwd(c["x"], c["a"], sigmoid=sigmoid, init_state=c["init"], keep_states=True)
    want = oracle.scan_f64(c["x"], c["a"], sigmoid, c["init"])
    check_fwd(c, sigmoid, (y, final), want)
    assert rel(kept, torch.stack(want[1][:-1:bd.GATED_SCAN_KEEP], 1)) <= tol(F32, L)
    grads = oracle.scan_grads_f64(c["x"], c["a"], sigmoid, c["dy"], c["init"], c["d_final"])
    check_bwd(c, sigmoid, run_bwd(c, sigmoid, kept), grads, want[1])
    # without the kept states, and without the last state's gradient
    grads = oracle.scan_grads_f64(c["x"], c["a"], sigmoid, c["dy"], c["init"])
    check_bwd(c, sigmoid, run_bwd(c, sigmoid, d_final=False), grads, want[1])


@pytest.mark.parametrize("dtype,a_dtype", TYPES)
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("K", [1, 2, 5, 16])
def test_step(dtype, a_dtype, sigmoid, K):
    for D in (1, 63, 512, 1291):
        c = make(4, K, D, sigmoid, dtype, a_dtype, seed=K + D)
        accept = torch.tensor([0, K, K // 2, 1], dtype=torch.int32, device="cuda")
        y, state = bd.gated_scan_step(c["init"], c["x"], c["a"], sigmoid=sigmoid, accept_len=accept)
        ey, states = oracle.scan_f64(c["x"], c["a"], sigmoid, c["init"])
        assert rel(y, ey) <= tol(dtype, K)
        assert torch.equal(state[0], c["init"][0])
        assert rel(state, torch.stack([states[int(n)][i] for i, n in enumerate(accept)])) <= tol(F32, K)
        _, last = bd.gated_scan_step(c["init"], c["x"], c["a"], sigmoid=sigmoid)
        assert torch.equal(last[1], state[1]) and rel(last, states[-1]) <= tol(F32, K)


def test_step_in_place_and_bad_counts():
    c = make(3, 4, 70, True, BF, BF, seed=1)
    y0, s0 = bd.gated_scan_step(c["init"], c["x"], c["a"], sigmoid=True)
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    accept = torch.tensor([4, 9, -3], dtype=torch.int32, device="cuda")
    state, y = c["init"].clone(), torch.empty_like(y0)
    bd.ssd_gated_scan_step(state, c["x"], c["a"], accept, y, state, True, flag)
    assert int(flag) == 1 and torch.equal(y, y0)
    assert torch.equal(state[:2], s0[:2]) and torch.equal(state[2], c["init"][2])
    flag.zero_()
    _, state = bd.gated_scan_step(c["init"], c["x"], c["a"], sigmoid=True, accept_len=accept.clamp(0, 4), err_flag=flag)
    assert int(flag) == 0


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prefill_then_decode(dtype):
    """A prompt through the sequence call, then tokens one and three at a time, against the whole."""
    c = make(2, 700, 90, True, dtype, dtype, seed=3)
    y, final = bd.gated_scan_fwd(c["x"], c["a"], sigmoid=True, init_state=c["init"])
    part = lambda lo, hi: (c["x"][:, lo:hi].contiguous(), c["a"][:, lo:hi].contiguous())
    _, state = bd.gated_scan_fwd(*part(0, 696), sigmoid=True, init_state=c["init"])
    for lo, hi in ((696, 697), (697, 700)):
        yt, state = bd.gated_scan_step(state, *part(lo, hi), sigmoid=True)
        assert rel(yt, y[:, lo:hi]) <= 2 * tol(dtype, 700)
    assert rel(state, final) <= 2 * tol(F32, 700)


@pytest.mark.parametrize("L", [0, 1])
def test_short_and_empty(L):
    c = make(2, L, 40, False, BF, F32, seed=1)
    y, final, kept = bd.gated_scan_fwd(c["x"], c["a"], init_state=c["init"], keep_states=True)
    assert y.shape == (2, L, 40) and kept.shape == (2, L, 40)
    if L == 0:
        assert torch.equal(final, c["init"])
        _, zero = bd.gated_scan_fwd(c["x"], c["a"])
        assert float(zero.abs().max()) == 0.0
    dx, da, d_init = run_bwd(c, False, kept)
    assert dx.shape == (2, L, 40)
    if L == 0:
        assert torch.equal(d_init, c["d_final"])
    e = torch.empty((0, 5, 8), device="cuda")
    y, final = bd.gated_scan_fwd(e, e)
    assert y.shape == (0, 5, 8) and final.shape == (0, 8)


@pytest.mark.parametrize("a", [0.0, -1e-7, -1e-6, -1e-5, -1e-3, -0.2, -0.2499, -0.25, -0.26, -5.0, -80.0])
def test_constant_gates(a):
    """Every token's gate is off in the same way: the error of its distance from 1 counts, not
    of its nearest 32-bit value.  beta is off by at most 4 U of itself (the series' rounding
    and that of a log2 e), which over the memory's length 1 / beta is 4 U of the state."""
    L, D = 4096, 64
    x = torch.rand((1, L, D), generator=torch.Generator().manual_seed(1)).cuda() + 0.5
    gate = torch.full((1, L, D), a, device="cuda")
    init = torch.full((1, D), 100.0, device="cuda")
    y, final = bd.gated_scan_fwd(x, gate, init_state=init)
    ey, states = oracle.scan_f64(x, gate, False, init)
    assert rel(y, ey) <= tol(F32, L) and rel(final, states[-1]) <= tol(F32, L)


@pytest.mark.parametrize("z", [30.0, 14.0, 7.0, 1.0, 1e-3, 0.0, -1e-3, -3.0, -30.0])
def test_constant_sigmoid_gates(z):
    """The state starts within the values, so that what moves it in a token goes below and
    above its last bit at random."""
    L, D = 4096, 64
    x = torch.rand((1, L, D), generator=torch.Generator().manual_seed(1)).cuda() + 0.5
    gate = torch.full((1, L, D), z, device="cuda")
    init = torch.full((1, D), 1.0, device="cuda")
    y, final = bd.gated_scan_fwd(x, gate, sigmoid=True, init_state=init)
    ey, states = oracle.scan_f64(x, gate, True, init)
    assert rel(y, ey) <= tol(F32, L) and rel(final, states[-1]) <= tol(F32, L)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("where", [1, 40, 300, 1999])
def test_erased_large_state(sigmoid, where):
    """A state 2^20 times the values, erased to 1e-4 of itself or wholly: what stays counts to
    24 bits of itself, and no more of the large one is left."""
    L, D = 2000, 64
    c = make(1, L, D, sigmoid, F32, F32, seed=4)
    c["a"][:] = 8.0 if sigmoid else -1e-3
    c["a"][:, where, :32] = math.log(1e-4)          # a sigmoid of it is 1e-4 / (1 + 1e-4)
    c["a"][:, where, 32:] = -math.inf
    c["init"] *= 2.0 ** 20
    y, final = bd.gated_scan_fwd(c["x"], c["a"], sigmoid=sigmoid, init_state=c["init"])
    ey, states = oracle.scan_f64(c["x"], c["a"], sigmoid, c["init"])
    for part in (slice(0, 32), slice(32, 64)):
        assert rel(y[:, where:, part], ey[:, where:, part]) <= tol(F32, L)
        assert rel(final[:, part], states[-1][:, part]) <= tol(F32, L)


def test_packed_sequences_and_padding():
    """a = -infinity at the first token of each of several sequences in one row; tokens with
    a = 0 and x = 0 at the end leave the state."""
    lens = [5, 300, 1, 77, 600]
    c = make(1, sum(lens), 48, False, BF, F32, seed=5, init=False)
    starts = [sum(lens[:i]) for i in range(len(lens))]
    c["a"][:, starts] = -math.inf
    y, _ = bd.gated_scan_fwd(c["x"], c["a"])
    dx, da, _ = bd.gated_scan_bwd(c["x"], c["a"], c["dy"])
    for at, n in zip(starts, lens):
        own = [c[k][:, at:at + n].contiguous() for k in ("x", "a", "dy")]
        own[1][:, 0] = -1.0
        yo, _ = bd.gated_scan_fwd(*own[:2])
        dxo, dao, _ = bd.gated_scan_bwd(*own)
        assert rel(y[:, at:at + n], yo) <= 2 * tol(BF, n) and rel(dx[:, at:at + n], dxo) <= 2 * tol(BF, n)
        assert rel(da[:, at + 1:at + n], dao[:, 1:]) <= 8 * tol(F32, n)
        assert float(da[:, at].abs().max()) == 0.0
    padded = [torch.cat((c[k][:, :300], torch.zeros_like(c[k][:, :500])), 1) for k in ("x", "a")]
    _, short = bd.gated_scan_fwd(c["x"][:, :300].contiguous(), c["a"][:, :300].contiguous())
    _, final = bd.gated_scan_fwd(*padded)
    assert rel(final, short) <= tol(F32, 300)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_nan_stays_in_its_channel_and_later_tokens(sigmoid):
    c = make(2, 1500, 130, sigmoid, BF, F32, seed=6)
    y0, f0 = bd.gated_scan_fwd(c["x"], c["a"], sigmoid=sigmoid, init_state=c["init"])
    g0 = run_bwd(c, sigmoid)
    c["x"][0, 700, 5] = float("nan")
    c["a"][1, 900, 6] = float("nan")
    c["init"][1, 129] = float("inf")
    y, f = bd.gated_scan_fwd(c["x"], c["a"], sigmoid=sigmoid, init_state=c["init"])
    assert torch.equal(y[0, :700], y0[0, :700]) and torch.isnan(y[0, 700:, 5]).all() and torch.isnan(f[0, 5])
    assert torch.equal(y[1, :900, :129], y0[1, :900, :129]) and torch.isnan(y[1, 900:, 6]).all()
    assert not torch.isfinite(y[1, 0, 129])
    rest = torch.ones(2, 130, dtype=torch.bool, device="cuda")
    rest[0, 5] = rest[1, 6] = rest[1, 129] = False
    assert torch.equal(y.movedim(1, 2)[rest], y0.movedim(1, 2)[rest]) and torch.equal(f[rest], f0[rest])
    dx, da, di = run_bwd(c, sigmoid)
    for t, t0 in ((dx, g0[0]), (da, g0[1])):
        assert torch.equal(t.movedim(1, 2)[rest], t0.movedim(1, 2)[rest])
    assert torch.equal(di[rest], g0[2][rest])
    # gradients run the other way: those of tokens behind a NaN in the gate are as they were
    assert torch.equal(dx[1, 900:, 6] if not sigmoid else dx[1, 901:, 6], g0[0][1, 900:, 6] if not sigmoid else g0[0][1, 901:, 6])
    assert torch.isnan(da[1, 900, 6]) and (sigmoid or torch.isnan(dx[1, :900, 6]).all())


def test_results_repeat():
    for sigmoid in (False, True):
        c = make(3, 4001, 322, sigmoid, BF, BF, seed=7)
        first = bd.gated_scan_fwd(c["x"], c["a"], sigmoid=sigmoid, init_state=c["init"], keep_states=True) + run_bwd(c, sigmoid)
        for _ in range(5):
            again = bd.gated_scan_fwd(c["x"], c["a"], sigmoid=sigmoid, init_state=c["init"], keep_states=True) + run_bwd(c, sigmoid)
            assert all(torch.equal(s, t) for s, t in zip(first, again))


def test_rows_behind_the_last_stay():
    c = make(1, 300, 66, False, BF, F32, seed=8)
    y, dx = (torch.full((1, 310, 66), 7.0, dtype=BF, device="cuda") for _ in range(2))
    da = torch.full((1, 310, 66), 7.0, device="cuda")
    kept = torch.full((1, 12, 66), 7.0, device="cuda")
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    bd.ssd_gated_scan_fwd(c["x"], c["a"], c["init"], y[:, :300], kept[:, :10], None, False, ws)
    bd.ssd_gated_scan_bwd(c["x"], c["a"], None, kept[:, :10], c["dy"], None, dx[:, :300], da[:, :300], None, False, ws)
    torch.cuda.synchronize()
    assert all(bool((t == 7.0).all()) for t in (y[:, 300:], dx[:, 300:], da[:, 300:], kept[:, 10:]))
    assert bool((y[:, :300] != 7.0).any())


@pytest.mark.parametrize("L", [20, 300, 3000])
def test_captured_and_replayed(L):
    b, D = 2, 96
    c = make(b, L, D, True, BF, BF, seed=21)
    n = max(bd.ssd_gated_scan_fwd_workspace_bytes(b, L, D, bd.SSD_DTYPE_BF16, bd.SSD_DTYPE_BF16),
            bd.ssd_gated_scan_bwd_workspace_bytes(b, L, D, False, bd.SSD_DTYPE_BF16, bd.SSD_DTYPE_BF16))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    y, dx, da = (torch.empty_like(c["x"]) for _ in range(3))
    final, d_init = torch.empty_like(c["init"]), torch.empty_like(c["init"])
    outs = [y, final, dx, da, d_init]

    def step():
        bd.ssd_gated_scan_fwd(c["x"], c["a"], c["init"], y, None, final, True, ws)
        bd.ssd_gated_scan_bwd(c["x"], c["a"], c["init"], None, c["dy"], c["d_final"], dx, da, d_init, True, ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        c["x"].copy_(make(b, L, D, True, BF, BF, seed=30 + seed)["x"])
        ws.fill_(seed * 85)         # a workspace needs no preparation
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        for t in outs:
            t.zero_()
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(s, t) for s, t in zip(got, outs))


def test_two_streams_at_once():
    """Two calls in flight, each with a workspace of its own, repeat what each gives alone."""
    cs = [make(2, 3000, 640, False, BF, F32, seed=s) for s in (1, 2)]
    want = [bd.gated_scan_fwd(c["x"], c["a"], init_state=c["init"]) + run_bwd(c, False) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    got = [bd.gated_scan_fwd(c["x"], c["a"], init_state=c["init"], stream=s)
           + bd.gated_scan_bwd(c["x"], c["a"], c["dy"], init_state=c["init"], d_final=c["d_final"], stream=s) for c, s in zip(cs, streams)]
    for s in streams:
        s.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(s, t) for s, t in zip(g, w))


def test_binding_refusals():
    c = make(1, 8, 16, False, BF, F32)
    with pytest.raises(TypeError):
        bd.gated_scan_fwd(c["x"].half(), c["a"])
    with pytest.raises(bd.SSDError):            # fp32 values with a bf16 gate
        bd.gated_scan_fwd(c["x"].float(), c["a"].to(BF))
    with pytest.raises(ValueError):
        bd.gated_scan_fwd(c["x"], c["a"][:, :7].contiguous())
    with pytest.raises(ValueError):
        bd.gated_scan_fwd(c["x"].transpose(1, 2), c["a"].transpose(1, 2))
    with pytest.raises(ValueError):
        bd.gated_scan_bwd(c["x"], c["a"], c["dy"], states=torch.zeros(1, 2, 16, device="cuda"))
