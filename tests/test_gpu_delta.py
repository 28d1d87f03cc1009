"""The gated delta rule against its float64 recurrence (MI355X only).

States are carried in 32 bits in both types, y is rounded once: tolerances in
delta_helpers.  With bfloat16 the outputs y may be formed from operands rounded to
bfloat16 (the state, the scores and the update: 3 roundings, and y's own).
"""
import math

import pytest
import torch

from delta_helpers import CUT, MANY, U32, inputs_of, make, rel, tol32, tol_out
from oracle import delta
from selective_state_space_ssd_amd import binding as bd

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def check_fwd(c, scale, L, N, dtype, amplified=1.0):
    y, S = bd.gated_delta_fwd(*inputs_of(c), scale, init_state=c["init_state"])
    ey, es = delta.delta_f64(*inputs_of({n: t if t is None else t.cpu() for n, t in c.items()}), scale,
                             None if c["init_state"] is None else c["init_state"].cpu())
    assert y.dtype == dtype and S.dtype == F32
    assert rel(y, ey) <= tol_out(dtype, L, N, 4) + (amplified - 1) * tol32(L, N)
    assert rel(S, es[-1]) <= amplified * tol32(L, N)
    return y, S


# b, L, H, G, P, N: lengths of one, about the chunk of 64 and beyond; one head per group
# and several; head sizes that no tile divides; every state width
FWD = [(1, 1, 1, 1, 16, 16), (2, 3, 4, 2, 16, 32), (1, 16, 2, 1, 32, 32), (1, 17, 2, 1, 32, 32), (2, 63, 2, 2, 64, 64), (1, 64, 4, 1, 64, 64),
       (1, 65, 3, 1, 48, 64), (2, 128, 2, 1, 128, 128), (1, 193, 6, 2, 96, 128), (1, 130, 2, 1, 80, 128), (1, 150, 2, 2, 64, 256), (1, 200, 2, 1, 256, 256),
       (3, 77, 5, 5, 16, 64), (1, 70, 2, 1, 20, 64), (1, 40, 2, 1, 1, 128), (1, 300, 1, 1, 33, 32), (1, 100, 3, 1, 64, 16)]


@pytest.mark.parametrize("b,L,H,G,P,N", FWD)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("init", [False, True])
def test_sequence(b, L, H, G, P, N, dtype, init):
    check_fwd(make(b, L, H, G, P, N, dtype, seed=L + N, init=init), N ** -0.5, L, N, dtype)


@pytest.mark.parametrize("b,L,H,G,P,N", MANY)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_heads_or_chunks(b, L, H, G, P, N, dtype):
    check_fwd(make(b, L, H, G, P, N, dtype, seed=L + N), N ** -0.5, L, N, dtype)


@pytest.mark.parametrize("L", [16, 17, 24, 25, 32, 33])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_where_chunks_begin(L, dtype):
    check_fwd(make(2, L, 4, 2, 48, 64, dtype, seed=L), 0.125, L, 64, dtype)


def test_long_sequence():
    c = make(1, 1500, 2, 1, 64, 128, BF, seed=5)
    check_fwd(c, 1.0, 1500, 128, BF)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_state_handed_on(dtype):
    """Two halves with the state handed on give the whole."""
    c = make(2, 150, 4, 2, 64, 64, dtype, seed=9)
    y, S = bd.gated_delta_fwd(*inputs_of(c), 0.5, init_state=c["init_state"])
    cut = 87
    first = [t[:, :cut].contiguous() for t in inputs_of(c)]
    rest = [t[:, cut:].contiguous() for t in inputs_of(c)]
    y1, S1 = bd.gated_delta_fwd(*first, 0.5, init_state=c["init_state"])
    y2, S2 = bd.gated_delta_fwd(*rest, 0.5, init_state=S1)
    assert rel(S2, S) <= 2 * tol32(150, 64)
    assert rel(torch.cat([y1, y2], 1), y) <= 2 * tol_out(dtype, 150, 64, 4)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("L", [10, 100])
def test_gates_at_their_ends(dtype, L):
    """Tokens that forget everything (a = -inf, the type's lowest value, -1e4), that keep
    everything (a = 0), that write nothing (beta = 0), that replace (beta = 1)."""
    c = make(1, L, 4, 2, 32, 64, dtype, seed=3)
    c["a"][:, 2, 0] = -math.inf
    c["a"][:, 5, 1] = torch.finfo(F32).min
    c["a"][:, 7, 2] = -1e4
    c["a"][:, ::3, 3] = -math.inf
    c["a"][:, 4:, 2] = 0.0
    c["beta"][:, 3:, 1] = 0.0
    c["beta"][:, ::2, 0] = 1.0
    y, S = check_fwd(c, 0.3, L, 64, dtype)
    assert torch.isfinite(y).all() and torch.isfinite(S).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_equal_keys(dtype):
    """One key over and over with beta = 1, no decay: the state holds the last value; the
    triangular system of a chunk is as badly scaled as the domain allows."""
    c = make(1, 140, 2, 1, 32, 64, dtype, seed=4, init=False)
    c["k"][:] = 0.0
    c["k"][..., 3] = 1.0
    c["a"].zero_()
    c["beta"].fill_(1.0)
    _, S = check_fwd(c, 1.0, 140, 64, dtype)
    assert rel(S[0, :, :, 3], c["v"][0, -1].float()) <= tol32(140, 64)
    # the far end, every update reflects.  In a chunk of 64, E_i = R_i + sum_j M_ij beta_j R_j
    # with R the brackets at the chunk's start.  For one unit key k_i . k_j = 1 and Lo is all
    # ones below the diagonal, so (I + 2 Lo) M = -Lo has M_ij = (-1)^(i - j): every weight
    # M_ij beta_j is 2 or -2.  The brackets' independent errors of one rounding each come out
    # 2 sqrt(63) < 16 times as large, while E, the bracket itself, does not grow: the token
    # by token form reflects, |E_i| <= |v_i| + |w|
    c["beta"].fill_(2.0)
    check_fwd(c, 1.0, 140, 64, dtype, amplified=16.0)


def test_padded_tokens_change_nothing():
    c = make(2, 100, 2, 1, 64, 64, BF, seed=6)
    n = 71
    c["a"][1, n:] = 0.0
    c["beta"][1, n:] = 0.0
    _, S = bd.gated_delta_fwd(*inputs_of(c), 1.0, init_state=c["init_state"])
    short = [t[1:, :n].contiguous() for t in inputs_of(c)]
    _, S1 = bd.gated_delta_fwd(*short, 1.0, init_state=c["init_state"][1:].contiguous())
    assert rel(S[1:], S1) <= tol32(100, 64)


def test_heads_apart_from_nan_in_others_and_later_tokens():
    c = make(1, 130, 4, 2, 32, 64, BF, seed=8)
    y0, S0 = bd.gated_delta_fwd(*inputs_of(c), 1.0, init_state=c["init_state"])
    c["v"][0, 100, 1, 5] = float("nan")
    y, S = bd.gated_delta_fwd(*inputs_of(c), 1.0, init_state=c["init_state"])
    keep = [0, 2, 3]
    assert torch.equal(y[:, :, keep], y0[:, :, keep]) and torch.equal(S[:, keep], S0[:, keep])
    assert torch.equal(y[:, :64], y0[:, :64])          # earlier chunks
    assert y[0, 100, 1, 5].isnan() and S[0, 1, 5].isnan().all()
    assert torch.equal(S[0, 1, :5], S0[0, 1, :5])


def test_no_tokens_and_no_rows():
    c = make(2, 0, 2, 1, 16, 32, BF)
    y, S = bd.gated_delta_fwd(*inputs_of(c), 1.0, init_state=c["init_state"])
    assert y.shape == (2, 0, 2, 16) and torch.equal(S, c["init_state"])
    _, S = bd.gated_delta_fwd(*inputs_of(c), 1.0)
    assert float(S.abs().max()) == 0.0
    c = make(0, 5, 2, 1, 16, 32, BF)
    y, S = bd.gated_delta_fwd(*inputs_of(c), 1.0)
    assert y.shape == (0, 5, 2, 16) and S.shape == (0, 2, 16, 32)


def test_without_final_state_and_rows_behind_stay():
    c = make(1, 90, 2, 1, 64, 64, BF, seed=2)
    y0, _ = bd.gated_delta_fwd(*inputs_of(c), 1.0, init_state=c["init_state"])
    big = torch.full((2, 90, 2, 64), 7.0, dtype=BF, device="cuda")
    n = bd.ssd_gated_delta_fwd_workspace_bytes(1, 90, 2, 64, 64, 1, bd.SSD_DTYPE_BF16)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    bd.ssd_gated_delta_fwd(*inputs_of(c), c["init_state"], big[:1], None, 1.0, ws)
    assert torch.equal(big[:1], y0) and (big[1] == 7.0).all()


@pytest.mark.parametrize("b,K,H,G,P,N", [(1, 1, 1, 1, 1, 16), (3, 1, 4, 2, 64, 128), (2, 5, 4, 1, 40, 64), (2, 16, 2, 2, 128, 128), (5, 3, 6, 3, 100, 256), (4, 2, 2, 1, 33, 32)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_step(b, K, H, G, P, N, dtype):
    c = make(b, K, H, G, P, N, dtype, seed=K)
    cpu = {n: t.cpu() for n, t in c.items()}
    ey, es = delta.delta_f64(*inputs_of(cpu), 0.7, cpu["init_state"])
    y, S = bd.gated_delta_step(c["init_state"], *inputs_of(c), 0.7)
    # y is a sum of N products S q: its error in 32 bits goes by the products' size (an
    # fp32 sum is off by at most N 2^-24 sum |S q|), and a single y may be far smaller
    # than they are; its one rounding to the type goes by y itself
    r = H // G
    terms = 0.7 * torch.stack([(s.abs() * cpu["q"][:, t].double().abs().repeat_interleave(r, 1)[:, :, None]).sum(-1) for t, s in enumerate(es[1:])], 1)
    rounded = 0.0 if dtype == F32 else torch.finfo(dtype).eps / 2 * float(ey.norm())
    assert float((y.double().cpu() - ey).norm()) <= rounded + tol32(K, N) * float(terms.norm())
    assert rel(S, es[-1]) <= tol32(K, N)
    acc = torch.tensor([i % (K + 1) for i in range(b)], dtype=torch.int32, device="cuda")
    y2, S2 = bd.gated_delta_step(c["init_state"], *inputs_of(c), 0.7, accept_len=acc)
    assert torch.equal(y2, y)
    for i in range(b):
        n = int(acc[i])
        assert torch.equal(S2[i], c["init_state"][i]) if n == 0 else rel(S2[i], es[n][i]) <= tol32(K, N)


def test_step_in_place_and_bad_counts():
    c = make(3, 4, 2, 1, 64, 64, BF, seed=1)
    y0, S0 = bd.gated_delta_step(c["init_state"], *inputs_of(c), 1.0)
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    acc = torch.tensor([4, 9, -3], dtype=torch.int32, device="cuda")
    S, y = c["init_state"].clone(), torch.empty_like(y0)
    bd.ssd_gated_delta_step(S, *inputs_of(c), acc, y, S, 1.0, err_flag=flag)
    assert int(flag) == 1 and torch.equal(y, y0)
    assert torch.equal(S[:2], S0[:2]) and torch.equal(S[2], c["init_state"][2])


def test_prefill_then_decode():
    """A prompt through the sequence call, then tokens one at a time, against the whole."""
    c = make(2, 100, 4, 2, 64, 64, BF, seed=13)
    y, S = bd.gated_delta_fwd(*inputs_of(c), 0.5, init_state=c["init_state"])
    n = 96
    part = [t[:, :n].contiguous() for t in inputs_of(c)]
    _, state = bd.gated_delta_fwd(*part, 0.5, init_state=c["init_state"])
    for t in range(n, 100):
        yt, state = bd.gated_delta_step(state, *[x[:, t:t + 1].contiguous() for x in inputs_of(c)], 0.5)
        assert rel(yt, y[:, t:t + 1]) <= 2 * tol_out(BF, 100, 64, 4)
    assert rel(state, S) <= 2 * tol32(100, 64)


@pytest.mark.parametrize("L", [8, 200, 2000])
def test_captured_and_replayed(L):
    c = make(2, L, 4, 2, 64, 128, BF, seed=21)
    n = bd.ssd_gated_delta_fwd_workspace_bytes(2, L, 4, 64, 128, 2, bd.SSD_DTYPE_BF16)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    y, S = torch.empty_like(c["v"]), torch.empty_like(c["init_state"])

    def step():
        bd.ssd_gated_delta_fwd(*inputs_of(c), c["init_state"], y, S, 0.5, ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        c["v"].copy_(make(2, L, 4, 2, 64, 128, BF, seed=30 + seed)["v"])
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone(), S.clone()
        y.zero_()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got[0], y) and torch.equal(got[1], S)


def test_two_streams_at_once():
    """Two calls in flight, each with a workspace of its own, repeat what each gives alone."""
    cs = [make(1, 700, 4, 2, 64, 128, BF, seed=s) for s in (1, 2)]
    want = [bd.gated_delta_fwd(*inputs_of(c), 0.5, init_state=c["init_state"]) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    got = [bd.gated_delta_fwd(*inputs_of(c), 0.5, init_state=c["init_state"], stream=s) for c, s in zip(cs, streams)]
    for s in streams:
        s.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


@pytest.mark.parametrize("b,L,H,G,P,N", CUT)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("init", [False, True])
def test_cut_into_segments(b, L, H, G, P, N, dtype, init):
    if N >= 32 and (N < 256 or dtype == BF):    # the workspace holds more than each chunk's image: the segments' states
        of = lambda tokens: bd.ssd_gated_delta_fwd_workspace_bytes(b, tokens, H, P, N, G, bd.SSD_DTYPE_BF16 if dtype == BF else bd.SSD_DTYPE_F32)
        assert of(L) > of(128) // 2 * ((L + 63) // 64)
    check_fwd(make(b, L, H, G, P, N, dtype, seed=L + N, init=init), N ** -0.5, L, N, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_cut_reflections_and_closed_gates(dtype):
    """beta = 2 (the map of a segment is a reflection after the other, which shortens no
    state) and a gate that closes in the middle (it is 0 from there on)."""
    c = make(1, 1500, 2, 1, 32, 64, dtype, seed=4)
    c["beta"][:, :, 0] = 2.0
    c["a"][:, :, 0] = 0.0
    c["a"][:, 700, 1] = -float("inf")
    # as in test_equal_keys: M_ij beta_j is what token i reads of the reflections of 2 k_j, at
    # most 2, so that a chunk's brackets take up 2 sqrt(63) < 16 times one rounding's error;
    # the map from segment to segment is an isometry
    check_fwd(c, 0.5, 1500, 64, dtype, amplified=16)


def test_cut_rows_apart_from_nan_in_others():
    c = make(1, 2000, 2, 1, 64, 128, BF, seed=2)
    y, S = bd.gated_delta_fwd(*inputs_of(c), 1.0, init_state=c["init_state"])
    c["v"][:, 1100, 0, 5] = float("nan")
    c["init_state"][:, 1, 7] = float("inf")
    y2, S2 = bd.gated_delta_fwd(*inputs_of(c), 1.0, init_state=c["init_state"])
    keep = torch.ones(2, 64, dtype=torch.bool, device="cuda")
    keep[0, 5] = keep[1, 7] = False
    assert torch.equal(y2[:, :, keep], y[:, :, keep]) and torch.equal(S2[:, keep], S[:, keep])
    assert torch.equal(y2[:, :1088, 0], y[:, :1088, 0])        # earlier chunks
    assert torch.isnan(y2[:, 1100:, 0, 5]).all() and not torch.isfinite(S2[:, 1, 7]).any()
