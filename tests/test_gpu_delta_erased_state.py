"""The gated delta rule where its updates erase what the state held: y is then far smaller
than the terms that it is a sum of (MI355X only).

The first 32 keys are orthogonal with beta |k|^2 = 1, so that they replace a state of N = 32
columns whole, and they come again: of a large state that enters, nothing is left after 32
tokens, in the middle of a chunk.  Gates are open (a = 0).  All inputs are whole numbers
and powers of two, so that the products and sums of 32 bits are exact.
"""
import pytest
import torch

from delta_helpers import inputs_of
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
