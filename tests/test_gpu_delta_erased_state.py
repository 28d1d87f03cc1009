"""The gated delta rule where its updates erase what the state held: y and the gradients are
then far smaller than the terms that they are sums of (MI355X only).

The first 32 keys are orthogonal with beta |k|^2 = 1, so that they replace a state of N = 32
columns whole, and they come again: of a large state that enters, nothing is left after 32
tokens, in the middle of a chunk.  Gates are open (a = 0).  All inputs are whole numbers
and powers of two, so that the products and sums of 32 bits are exact, or nearly so.

Tolerance of the gradients, per token, of 2-norms: the output's own rounding, half a step of
its type, and 16 x 2^-24 of the terms' size.  The terms (of dq: dy S; of dk: dv S and u dS;
of dv: k dS) pass at most 16 roundings of 32 bits, each 2^-24 of a partial sum no larger than
they are: the product with the state (in up to 6 products of planes), the bracket, the product
with M (6) and beta, then the sum that the output is (up to 6).
"""
import math

import pytest
import torch

from delta_helpers import U32, inputs_of
from oracle import delta
from selective_state_space_ssd_amd import binding as bd

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
N = 32


def hadamard(n):
    h = torch.ones(1, 1)
    while h.shape[0] < n:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h


def make(L, H, P, dtype, entering, leaving, seed):
    """Keys +-1/4 (|k|^2 = 2) with beta = 1/2, whole-number queries, values and gradients of
    size 1; the states that enter forward (init_state) and backward (d_final) are whole
    numbers up to `entering` and `leaving`."""
    g = torch.Generator().manual_seed(seed)
    small = lambda *s: torch.randint(-1, 2, s, generator=g).float()
    large = lambda most, *s: torch.randint(-most, most + 1, s, generator=g).float()
    c = dict(q=small(1, L, 1, N), k=(hadamard(N) / 4)[torch.arange(L) % N].view(1, L, 1, N), v=small(1, L, H, P), dy=small(1, L, H, P))
    c = {n: t.to(dtype) for n, t in c.items()}
    c.update(a=torch.zeros(1, L, H), beta=torch.full((1, L, H), 0.5), init_state=large(entering, 1, H, P, N), d_final=large(leaving, 1, H, P, N))
    return c


def on_gpu(c):
    return {n: t.cuda() for n, t in c.items()}


def check_tokens(name, got, want, terms, dtype):
    """Per token (dimension 1) against half a step of `want` and 16 x 2^-24 of `terms`."""
    err = (got.double().cpu() - want).flatten(2).norm(dim=-1)
    tol = torch.finfo(dtype).eps / 2 * want.flatten(2).norm(dim=-1) + 16 * U32 * terms
    worst = int((err / tol).argmax())
    assert (err <= tol).all(), (name, worst, float(err[0, worst]), float(tol[0, worst]))


@pytest.mark.parametrize("most", [1 << 7, 1 << 16])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("L,P", [(64, 16), (100, 48)])
def test_outputs_after_an_erased_state(L, P, dtype, most):
    """Queries with a single 1: y picks one column of the state.  All sums of 32 bits are
    exact: the state's entries are whole numbers below 2^17, K S^T is in quarters and below
    2^19, U in eighths and below 2^18, scores U in thirty-seconds and, for these inputs, below
    2^18: 23 bits.  What is left is y's own rounding: half a step of its type."""
    c = make(L, 2, P, dtype, most, 1, seed=L + P)
    g = torch.Generator().manual_seed(1)
    c["q"] = torch.nn.functional.one_hot(torch.randint(0, N, (1, L, 1), generator=g), N).to(dtype)
    d = on_gpu(c)
    y, S = bd.gated_delta_fwd(*inputs_of(d), 1.0, init_state=d["init_state"])
    ey, es = delta.delta_f64(*inputs_of(c), 1.0, c["init_state"])
    assert torch.equal(S.double().cpu(), es[-1])
    err = (y.double().cpu() - ey).abs()
    assert (err <= torch.finfo(dtype).eps / 2 * ey.abs()).all(), (int((err - torch.finfo(dtype).eps / 2 * ey.abs()).flatten(2).amax(-1).argmax()), float(err.max()))


SIZES = [1 << 7, 1 << 13]


@pytest.mark.parametrize("most", SIZES)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("large", ["entering", "leaving"])
@pytest.mark.parametrize("L,P", [(64, 16), (100, 48)])
def test_gradients_beside_an_erased_state(L, P, large, dtype, most):
    c = make(L, 2, P, dtype, most if large == "entering" else 1, most if large == "leaving" else 1, seed=L + P)
    d = on_gpu(c)
    got = bd.gated_delta_bwd(*inputs_of(d), 1.0, d["dy"], init_state=d["init_state"], d_final=d["d_final"])
    want = delta.delta_grads_f64(*inputs_of(c), 1.0, c["dy"], c["init_state"], c["d_final"])
    S, dS, dv = c["init_state"].double(), c["d_final"].double(), want[2]
    _, states = delta.delta_f64(*inputs_of(c), 1.0, c["init_state"])
    prev = torch.stack(states[:-1], 1)
    k = c["k"].double().expand(1, L, 2, N)
    u = c["beta"].double()[..., None] * (c["v"].double() - (prev @ k[..., None])[..., 0])
    row = lambda x: x.double().flatten(2).norm(dim=-1).amax()
    # every product the sums are taken over: the state's, and those of the chunk's updates,
    # each no larger than the largest update times the largest gradient
    check_tokens("dq", got[0], want[0], row(c["dy"]) * (S.norm() + math.sqrt(L) * row(u) * row(k)), dtype)
    check_tokens("dk", got[1], want[1], row(dv) * S.norm() + row(u) * dS.norm() + math.sqrt(L) * row(u) * (row(dv) + row(c["dy"]) * row(c["q"])), dtype)
    check_tokens("dv", got[2], want[2], dS.norm() * row(k) + math.sqrt(L) * row(c["dy"]) * row(c["q"]), dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_gradients_of_reflections(dtype):
    """One unit key over and over with beta = 2 and open gates: every update reflects.  As in
    the forward test of equal keys, M_ij beta_j is 2 or -2 over a chunk: the brackets' errors
    of one rounding each come out up to 2 sqrt(63) < 16 times as large, and those of X, from
    the transposed system, too.  Tolerance: that, of the outputs' own terms."""
    L, H, P = 140, 2, 32
    g = torch.Generator().manual_seed(4)
    r = lambda *s: torch.randn(s, generator=g)
    c = dict(q=torch.nn.functional.normalize(r(1, L, 1, N), dim=-1).to(dtype), k=torch.zeros(1, L, 1, N, dtype=dtype), v=r(1, L, H, P).to(dtype),
             a=torch.zeros(1, L, H), beta=torch.full((1, L, H), 2.0), dy=r(1, L, H, P).to(dtype), init_state=0.1 * r(1, H, P, N), d_final=r(1, H, P, N))
    c["k"][..., 3] = 1.0
    d = on_gpu(c)
    got = bd.gated_delta_bwd(*inputs_of(d), 1.0, d["dy"], init_state=d["init_state"], d_final=d["d_final"])
    want = delta.delta_grads_f64(*inputs_of(c), 1.0, c["dy"], c["init_state"], c["d_final"])
    for name, x, w in zip(("dq", "dk", "dv", "da", "dbeta", "d_init"), got, want):
        half = torch.finfo(x.dtype).eps / 2
        err = float((x.double().cpu() - w).norm())
        # 16 roundings of 32 bits, 16 times as large twice over: E's and X's meet in dk, da, dbeta
        assert err <= (half + 2 * 16 * 16 * U32) * float(w.norm()), (name, err / float(w.norm()))
