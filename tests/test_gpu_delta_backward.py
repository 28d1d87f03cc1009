"""Gradients of the gated delta rule against the float64 gradients of its recurrence
(MI355X only).

da, dbeta and d_init are carried in 32 bits in both types.  With bfloat16, dq, dk and dv
are rounded once; the states and dv enter dq and dk rounded to bfloat16 as stored, each
once per product: up to 4 roundings.  da is a sum over up to 128 tokens of differences of
terms whose errors are those of 32-bit sums; it is compared with the terms' size.
"""
import math

import pytest
import torch

from delta_helpers import CUT, MANY, U32, inputs_of, make, rel, tol32, tol_out
from oracle import delta
from selective_state_space_ssd_amd import binding as bd

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NAMES = ("dq", "dk", "dv", "da", "dbeta", "d_init")


def cpu(c):
    return {n: t if t is None else t.cpu() for n, t in c.items()}


def gate_terms(c, scale):
    """2-norm, per token, of what da's formula adds up: y . dy and v . dv of the tokens up to
    128 further on, and <dS, S> at the segment's end, each with its elements' absolute values."""
    x = cpu(c)
    y, states = delta.delta_f64(*inputs_of(x), scale, x["init_state"])
    dv = delta.delta_grads_f64(*inputs_of(x), scale, x["dy"], x["init_state"], x["d_final"])[2]
    per_token = ((y * x["dy"].double()) ** 2).sum(-1) + ((dv * x["v"].double()) ** 2).sum(-1)
    end = ((states[-1] * x["d_final"].double()) ** 2).sum((-1, -2)) if x["d_final"] is not None else 0.0
    L = y.shape[1]
    out = torch.zeros_like(per_token)
    for t in range(L):
        out[:, t] = per_token[:, t:min(L, t + 128)].sum(1) + end
    return float(out.sum().sqrt())


def check(c, scale, L, N, dtype, amplified=1.0):
    got = bd.gated_delta_bwd(*inputs_of(c), scale, c["dy"], init_state=c["init_state"], d_final=c["d_final"])
    x = cpu(c)
    want = delta.delta_grads_f64(*inputs_of(x), scale, x["dy"], x["init_state"], x["d_final"])
    for name, g, w in zip(NAMES, got, want):
        assert g.dtype == (dtype if name in ("dq", "dk", "dv") else F32)
        # the backward pass runs on the forward's values: the errors of both
        tol = 2 * amplified * tol32(L, N)
        if name in ("dq", "dk", "dv") and dtype == BF:
            tol += (4 if name != "dv" else 1) * torch.finfo(dtype).eps / 2
        if name == "da":
            err = float((g.double().cpu() - w).norm())
            assert err <= tol * max(float(w.norm()), gate_terms(c, scale)), (name, err, float(w.norm()))
        else:
            assert rel(g, w) <= tol, (name, rel(g, w), tol)
    return got


# lengths of one, about the chunk (64) and the segment (128) and beyond; heads per group;
# head sizes that blocks of 32 and 64 rows do not divide; every state width
CASES = [(1, 1, 1, 1, 16, 32), (2, 5, 4, 2, 16, 32), (1, 63, 2, 1, 32, 64), (1, 64, 2, 2, 64, 64), (2, 65, 3, 1, 48, 64), (1, 130, 4, 2, 64, 128),
         (1, 200, 2, 1, 128, 128), (1, 256, 1, 1, 16, 32), (1, 257, 2, 1, 80, 32), (2, 330, 2, 1, 32, 64), (1, 100, 5, 5, 96, 32), (1, 90, 6, 1, 16, 64)]


@pytest.mark.parametrize("b,L,H,G,P,N", CASES)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("init", [False, True])
def test_gradients(b, L, H, G, P, N, dtype, init):
    check(make(b, L, H, G, P, N, dtype, seed=L + N, init=init), N ** -0.5, L, N, dtype)


@pytest.mark.parametrize("b,L,H,G,P,N", MANY)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_heads_or_chunks(b, L, H, G, P, N, dtype):
    if N == 256 and dtype == F32:
        pytest.skip("fp32 gradients go up to N = 128")
    check(make(b, L, H, G, P, N, dtype, seed=L + N), N ** -0.5, L, N, dtype)


@pytest.mark.parametrize("b,L,H,G,P,N", CUT)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("init", [False, True])
def test_cut_into_segments(b, L, H, G, P, N, dtype, init):
    if N == 256 and dtype == F32:
        pytest.skip("fp32 gradients go up to N = 128")
    c = make(b, L, H, G, P, N, dtype, seed=L + N, init=init)
    if not init:
        c["d_final"] = None
    check(c, N ** -0.5, L, N, dtype)


def test_widest_state():
    check(make(1, 140, 2, 1, 48, 256, BF, seed=3), 0.1, 140, 256, BF)


def test_largest_heads():
    check(make(1, 70, 1, 1, 256, 64, BF, seed=3), 0.3, 70, 64, BF)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_without_gradient_of_the_final_state(dtype):
    c = make(1, 150, 2, 1, 32, 64, dtype, seed=5)
    c["d_final"] = None
    check(c, 0.5, 150, 64, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_gates_at_their_ends(dtype):
    c = make(1, 140, 4, 2, 32, 64, dtype, seed=3)
    c["a"][:, 2, 0] = -math.inf
    c["a"][:, 70, 1] = torch.finfo(F32).min
    c["a"][:, 7, 2] = -1e4
    c["a"][:, ::3, 3] = -80.0
    c["beta"][:, 3:60, 1] = 0.0
    c["beta"][:, ::2, 0] = 1.0
    # a token that forgets everything passes no gradient to its gate; d/da of e^a at
    # -infinity is 0 where the float64 form would take 0 * infinity
    x = dict(c)
    x["a"] = c["a"].clamp(min=-1e5)
    got = bd.gated_delta_bwd(*inputs_of(c), 0.3, c["dy"], init_state=c["init_state"], d_final=c["d_final"])
    again = check(x, 0.3, 140, 64, dtype)
    for g, w in zip(got, again):
        assert torch.isfinite(g).all() and torch.equal(g, w)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_equal_keys(dtype):
    c = make(1, 140, 2, 1, 32, 64, dtype, seed=4)
    c["k"][:] = 0.0
    c["k"][..., 3] = 1.0
    c["a"].zero_()
    c["beta"].fill_(1.0)
    check(c, 1.0, 140, 64, dtype)


def test_against_differences():
    """Directional differences of the forward call itself, in fp32, over each input."""
    c = make(1, 80, 2, 1, 16, 32, F32, seed=7)
    grads = bd.gated_delta_bwd(*inputs_of(c), 1.0, c["dy"], init_state=c["init_state"], d_final=c["d_final"])

    def loss(x):
        y, S = bd.gated_delta_fwd(*inputs_of(x), 1.0, init_state=x["init_state"])
        return float((y.double() * c["dy"].double()).sum() + (S.double() * c["d_final"].double()).sum())

    g = torch.Generator().manual_seed(1)
    for name, d in zip(("q", "k", "v", "a", "beta", "init_state"), grads):
        way = torch.randn(c[name].shape, generator=g).cuda()
        h = 2.0 ** -8 * float(c[name].norm() / way.norm())
        up, down = dict(c), dict(c)
        up[name], down[name] = c[name] + h * way, c[name] - h * way
        slope = (loss(up) - loss(down)) / (2 * h)
        want = float((d.double() * way.double()).sum())
        # the third-order term of a step of 2^-8, and the rounding of the losses over 2 h
        scale = float(d.double().norm() * way.double().norm())
        size = float((c["dy"].double().norm() ** 2 + c["d_final"].double().norm() ** 2).sqrt())
        assert abs(slope - want) <= 2.0 ** -14 * scale + 64 * U32 * size / h


@pytest.mark.parametrize("dtype", [BF, F32])
def test_results_repeat_and_rows_behind_stay(dtype):
    c = make(1, 150, 4, 1, 64, 64, dtype, seed=8)
    one = bd.gated_delta_bwd(*inputs_of(c), 0.5, c["dy"], init_state=c["init_state"], d_final=c["d_final"])
    two = bd.gated_delta_bwd(*inputs_of(c), 0.5, c["dy"], init_state=c["init_state"], d_final=c["d_final"])
    assert all(torch.equal(x, y) for x, y in zip(one, two))
    big = [torch.full((2, *t.shape[1:]), 7.0, dtype=t.dtype, device="cuda") for t in one[:5]]
    ws = torch.empty(bd.ssd_gated_delta_bwd_workspace_bytes(1, 150, 4, 64, 64, 1, 1 if dtype == BF else 0), dtype=torch.uint8, device="cuda")
    bd.ssd_gated_delta_bwd(*inputs_of(c), c["init_state"], c["dy"], c["d_final"], *[t[:1] for t in big], None, 0.5, ws)
    for t, w in zip(big, one):
        assert torch.equal(t[:1], w) and (t[1] == 7.0).all()


def test_padded_tokens_get_no_gradient_of_others():
    c = make(2, 100, 2, 1, 32, 64, BF, seed=6)
    n = 71
    c["a"][1, n:] = 0.0
    c["beta"][1, n:] = 0.0
    c["dy"][1, n:] = 0.0
    got = bd.gated_delta_bwd(*inputs_of(c), 1.0, c["dy"], init_state=c["init_state"], d_final=c["d_final"])
    short = {k: (t[1:, :n] if k in ("q", "k", "v", "a", "beta", "dy") else t[1:]).contiguous() for k, t in c.items()}
    want = bd.gated_delta_bwd(*inputs_of(short), 1.0, short["dy"], init_state=short["init_state"], d_final=short["d_final"])
    for name, g, w in zip(NAMES, got, want):
        g = g[1:] if name == "d_init" else g[1:, :n]
        tol = 4 * tol32(100, 64) * (8 if name == "da" else 1)
        assert rel(g, w) <= tol + (torch.finfo(BF).eps if g.dtype == BF else 0), name
    assert float(got[2][1, n:].abs().max()) == 0.0


def test_no_tokens():
    c = make(2, 0, 2, 1, 16, 32, BF)
    got = bd.gated_delta_bwd(*inputs_of(c), 1.0, c["dy"], init_state=c["init_state"], d_final=c["d_final"])
    assert torch.equal(got[5], c["d_final"]) and got[0].shape == (2, 0, 1, 32)


@pytest.mark.parametrize("L", [150, 1600])
def test_captured_and_replayed(L):
    c = make(1, L, 4, 2, 64, 128, BF, seed=21)
    outs = [torch.empty_like(c[n]) for n in ("q", "k", "v", "a", "beta", "init_state")]
    ws = torch.empty(bd.ssd_gated_delta_bwd_workspace_bytes(1, L, 4, 64, 128, 2, bd.SSD_DTYPE_BF16), dtype=torch.uint8, device="cuda")

    def step():
        bd.ssd_gated_delta_bwd(*inputs_of(c), c["init_state"], c["dy"], c["d_final"], *outs, 0.5, ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        c["dy"].copy_(make(1, L, 4, 2, 64, 128, BF, seed=30 + seed)["dy"])
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, outs))


def test_a_block_of_a_model():
    """Rule, gated norm per head, residual sum and norm: forward and backward in a row, as a
    layer runs them, against float64."""
    from oracle import norms
    b, L, H, P, N, eps, scale = 2, 70, 4, 32, 64, 1e-5, 0.125
    c = make(b, L, H, 2, P, N, BF, seed=11, init=False)
    g = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(s, generator=g)
    z, w1 = r(b, L, H, P).to(BF).cuda(), (1 + 0.1 * r(P)).cuda()
    res, w2, ls = (2 * r(b, L, H * P)).cuda(), (1 + 0.1 * r(H * P)).cuda(), (0.5 + 0.1 * r(H * P)).cuda()
    dout, dsum = r(b, L, H * P).to(BF).cuda(), r(b, L, H * P).cuda()

    y, _ = bd.gated_delta_fwd(*inputs_of(c), scale)
    n = bd.norm_gate_fwd(y, z, w1, P, eps)
    out, total = bd.norm_add_fwd(n.view(b, L, H * P), res, w2, eps, scale=ls)
    dn, dres, dw2, dls = bd.norm_add_bwd(n.view(b, L, H * P), total, w2, dout, dsum, eps, scale=ls)
    dy, dz, dw1 = bd.norm_gate_bwd(y, z, w1, dn.view(b, L, H, P), P, eps)
    grads = bd.gated_delta_bwd(*inputs_of(c), scale, dy)

    # the same in float64 from end to end
    x = cpu(c)
    leaves = [x[k].double().requires_grad_() for k in ("q", "k", "v", "a", "beta")]
    y64, _ = delta._recurrence(*leaves, torch.zeros(b, H, P, N, dtype=torch.float64), scale)
    extra = [t.detach().double().cpu().requires_grad_() for t in (z, w1, res, w2, ls)]
    n64 = norms._gate(y64, extra[0], extra[1], P, eps, False)
    t64 = extra[2] + extra[4] * n64.reshape(b, L, H * P)
    o64 = norms._normed(t64, H * P, eps) * extra[3]
    want = torch.autograd.grad((o64 * dout.double().cpu()).sum() + (t64 * dsum.double().cpu()).sum(), leaves + extra)
    # bf16 values passed on: y, n, dn, dy (4) and the operands of the last stage (4)
    tol = 8 * torch.finfo(BF).eps / 2
    assert rel(out, o64.detach()) <= tol and rel(total, t64.detach()) <= tol
    for got, exp in zip(list(grads[:5]) + [dz, dw1, dres, dw2, dls], want):
        # gates and norm weights add differences of such values up: their roundings are
        # independent, the sums no smaller than the terms' mean
        assert rel(got, exp) <= 2 * tol
