"""The gradients of the gates of the gated delta rule, from open gates to closed ones, head
by head and token by token (MI355X only).

With S' the state after the decay and dS' its gradient, da_t = <dS'_t, S'_t> and S'_t =
e^{a_t} S_{t-1}: a gate that closes takes its own gradient down with it.  The tolerances go
by that gradient, not by the size of what the tokens around it contribute.
"""
import math

import pytest
import torch

from delta_helpers import CUT, U32, inputs_of, make, rel, tol32
from oracle import delta
from selective_state_space_ssd_amd import binding as bd

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def cpu(c):
    return {n: t if t is None else t.cpu() for n, t in c.items()}


def factors(c, scale):
    """S_{t-1} and dS'_t in float64, [b, L, H, P, N] each: the two factors of da_t / e^{a_t}."""
    q, k, v, a, beta = (c[n].double() for n in ("q", "k", "v", "a", "beta"))
    b, L, H, P = v.shape
    _, states = delta.delta_f64(q, k, v, a, beta, scale, c["init_state"])
    r = H // k.shape[2]
    k, q = k.repeat_interleave(r, 2), q.repeat_interleave(r, 2)
    dS = torch.zeros_like(states[0]) if c["d_final"] is None else c["d_final"].double()
    grads = []
    for t in reversed(range(L)):
        dS = dS + scale * c["dy"][:, t].double()[..., None] * q[:, t][:, :, None]
        back = beta[:, t][..., None] * (dS @ k[:, t][..., None])[..., 0]
        dS = dS - back[..., None] * k[:, t][:, :, None]
        grads.append(dS)
        dS = torch.exp(a[:, t])[..., None, None] * dS
    return torch.stack(states[:-1], 1), torch.stack(grads[::-1], 1)


def gates_of(c, scale):
    return bd.gated_delta_bwd(*inputs_of(c), scale, c["dy"], init_state=c["init_state"], d_final=c["d_final"])[3].double().cpu()


def tol(L, N, a):
    """Of da, relative to its size: the errors of S and dS, each a value carried in 32 bits,
    and of the decays, whose exponents (up to |a| for the pairs that count) are 32-bit."""
    return 2 * tol32(L, N) + 4 * abs(a) * U32


@pytest.mark.parametrize("a", [-0.01, -1.0, -2.0, -4.0, -8.0, -16.0])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("b,L,H,G,P,N", [(1, 200, 3, 1, 64, 64), (2, 65, 2, 2, 48, 128), (1, 130, 2, 1, 96, 32)])
def test_constant_gates(b, L, H, G, P, N, dtype, a):
    c = make(b, L, H, G, P, N, dtype, seed=L)
    c["a"].fill_(a)
    x = cpu(c)
    want = delta.delta_grads_f64(*inputs_of(x), N ** -0.5, x["dy"], x["init_state"], x["d_final"])[3]
    got = gates_of(c, N ** -0.5)
    for i in range(b):
        for h in range(H):
            assert rel(got[i, :, h], want[i, :, h]) <= tol(L, N, a), (i, h, rel(got[i, :, h], want[i, :, h]))


@pytest.mark.parametrize("b,L,H,G,P,N", CUT[1:4])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_strong_gates_in_long_sequences(b, L, H, G, P, N, dtype):
    """Sequences that are cut into segments; a gate per head, from -1 to -9."""
    c = make(b, L, H, G, P, N, dtype, seed=L)
    c["a"][:] = -1.0 - 8.0 * torch.arange(H, device="cuda") / H
    x = cpu(c)
    want = delta.delta_grads_f64(*inputs_of(x), 0.5, x["dy"], x["init_state"], x["d_final"])[3]
    got = gates_of(c, 0.5)
    for i in range(b):
        for h in range(H):
            assert rel(got[i, :, h], want[i, :, h]) <= tol(L, N, -9.0), (i, h)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_closed_gates_beside_open_ones(dtype):
    """Single tokens at -inf, the type's lowest value, -1e4, -80, -30 and -12 among ordinary
    ones: each da_t within its own factors' size, |e^{a_t}| |dS'_t| |S_{t-1}|; 0 where the
    decay is 0."""
    L, N = 150, 64
    c = make(1, L, 4, 2, 32, N, dtype, seed=3)
    closed = {(0, 2): -math.inf, (0, 63): -80.0, (0, 64): -30.0, (0, 149): -12.0, (1, 70): torch.finfo(F32).min, (1, 0): -80.0, (1, 128): -12.0, (2, 7): -1e4,
              (2, 8): -1e4, (2, 100): -30.0, (3, 127): -12.0, (3, 40): -80.0, (3, 41): -12.0}
    for (h, t), a in closed.items():
        c["a"][0, t, h] = a
    x = cpu(c)
    x["a"] = x["a"].clamp(min=-1e5)
    S, dS = factors(x, 0.3)
    want = torch.exp(x["a"].double()) * (S * dS).sum((-1, -2))
    size = torch.exp(x["a"].double()) * S.flatten(3).norm(dim=-1) * dS.flatten(3).norm(dim=-1)
    got = gates_of(c, 0.3)
    for (h, t), a in closed.items():
        err = abs(float(got[0, t, h] - want[0, t, h]))
        assert err <= tol(L, N, max(a, -100.0)) * float(size[0, t, h]) + 2.0 ** -126, (h, t, a, float(got[0, t, h]), float(want[0, t, h]))
        if a < -1000:
            assert float(got[0, t, h]) == 0.0
    # and of all tokens
    assert ((got - want).abs() <= 2 * tol(L, N, -100.0) * size + 2.0 ** -126).all()
