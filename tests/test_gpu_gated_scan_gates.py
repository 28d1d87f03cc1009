"""The gated scan's gates one by one: both sides of the border of a log decay's series (-1/16), a
wave's decays taken together on both sides of its borders (-1/16 and -1), both signs of a gate before
its sigmoid, in the forward pass and in the gradients; and every element of bf16 outputs (MI355X only).

U = 2^-24, half a step of 32 bits next to 1.  A log decay's alpha is off by
  - its series (-1/16 < a < 0): 4 U of beta = 1 - alpha, and what is made of it one rounding,
  - elsewhere: a unit in the last place of exp2 (2 U of alpha at the most) and |a| 2 U of alpha, from
    the rounding of a log2 e and of log2 e itself.
"""
import math

import pytest
import torch

from oracle import gated_scan as oracle
from scan_helpers import U, make, rel, tol
from selective_state_space_ssd_amd import binding as bd

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
N = 1 << 16


def spread(lo, hi, seed):
    """N gates between two bounds."""
    return (lo + (hi - lo) * torch.rand(N, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)).float().cuda()


def single(a, sigmoid=False, h=1.0):
    """One token with x = 0 on a state h, and its gradients where 1 reaches the state after it."""
    gate = a[None, None]
    x, one = torch.zeros_like(gate), torch.ones_like(gate)[0]
    y, final, kept = bd.gated_scan_fwd(x, gate, sigmoid=sigmoid, init_state=h * one, keep_states=True)
    dx, da, d_init = bd.gated_scan_bwd(x, gate, x, sigmoid=sigmoid, d_final=one, states=kept)
    ys, _ = bd.gated_scan_step(h * one, x, gate, sigmoid=sigmoid)
    assert torch.equal(ys, y) and torch.equal(final, y[:, 0])
    return y[0, 0].double(), dx[0, 0].double(), da[0, 0].double(), d_init[0].double()


@pytest.mark.parametrize("lo,hi", [(-1 / 16, 0.0), (-0.0625, -0.06), (-0.0630, -0.0625), (-0.1, -0.0625), (-1.0, -0.25), (-20.0, -1.0)])
def test_log_decays(lo, hi):
    a = spread(lo, hi, 1)
    alpha = a.double().exp()
    y, _, da, d_init = single(a)
    off = torch.where(a > -0.0625, 4 * U * (1 - alpha) + U, (2 + 2 * a.double().abs()) * U * alpha + U * alpha)
    for got in (y, d_init, da):         # da = lam alpha h, with lam = h = 1
        assert float(((got - alpha).abs() / off).max()) <= 1.0


def test_the_series_has_all_its_terms():
    """The mean error over 65536 gates, whose roundings go up and down alike: a result's is at most
    U / 2 and its mean's standard deviation U / 2 / sqrt(3 N), 2^-33.8; six of those and the first term
    left out, a^6 / 720 = 2^-33.5, are 2^-30.9.  The term before, a^5 / 120, would be 2^-27.3 at
    a = -0.058."""
    a = spread(-0.0625, -0.055, 2)
    y, _, _, d_init = single(a)
    alpha = a.double().exp()
    assert abs(float((y - alpha).mean())) <= 2.0 ** -30.9 and abs(float((d_init - alpha).mean())) <= 2.0 ** -30.9


@pytest.mark.parametrize("lo,hi", [(-1e-3, 1e-3), (-3.0, 3.0), (3.0, 17.0), (-17.0, -3.0), (17.0, 60.0), (-60.0, -17.0)])
def test_sigmoid_gates(lo, hi):
    """dx is beta itself.  The smaller of alpha and beta is off by |a| 2 U of itself from a log2 e and
    by 4 units from exp2, the sum and the reciprocal; the other one by U more."""
    a = spread(lo, hi, 3)
    alpha, beta = torch.sigmoid(a.double()), torch.sigmoid(-a.double())
    y, dx, da, d_init = single(a, True)
    least = (8 + 2 * a.double().abs()) * U * torch.minimum(alpha, beta)
    for got, want in ((y, alpha), (d_init, alpha), (dx, beta)):
        assert float(((got - want).abs() / (least + torch.where(want > 0.5, U, 0.0))).max()) <= 1.0
    # lam alpha beta (h - x): both factors' errors and two roundings
    want = alpha * beta
    assert float(((da - want).abs() / (want * (8 + 2 * a.double().abs() + 4) * U)).max()) <= 1.0


@pytest.mark.parametrize("total", [-1e-4, -0.0624, -0.0625, -0.0626, -0.3, -0.999, -1.0, -1.001, -4.0])
def test_decays_of_a_wave_together(total):
    """16 tokens whose log decays add up to about `total`, a different sum in each of the channels, and
    48 more with a = 0 and x = 0: the state behind them is the 16 taken together.  Down to -1 that is
    the gate of the sum, off by 15 roundings of sums (U |total| each) and as one gate; below the
    product, 16 gates and 15 roundings."""
    shares = torch.rand(16, N, generator=torch.Generator().manual_seed(5), dtype=torch.float64) + 0.5
    near = total * (1 + 1e-3 * (torch.rand(N, generator=torch.Generator().manual_seed(6), dtype=torch.float64) - 0.5))
    a = torch.zeros((1, 64, N), device="cuda")
    a[0, :16] = (shares / shares.sum(0) * near).float().cuda()
    x, one = torch.zeros_like(a), torch.ones((1, N), device="cuda")
    want = a.double().sum(1).exp()
    size = float(want.max())
    of_sum, of_product = 15 * abs(total) + 3 + 2 * abs(total) + 1, 16 * (3 + abs(total) / 4) + 15 + 1
    off = U * size * (of_sum if total * 1.0005 > -1 else max(of_sum, of_product))
    y, final = bd.gated_scan_fwd(x, a, init_state=one)
    for t in (16, 17, 40, 63):
        assert float((y[:, t].double() - want).abs().max()) <= off
    assert torch.equal(final, y[:, 63])
    # and backwards: the last 16 tokens' decays, seen by those before them
    back = a.flip(1).contiguous()
    dx, da, d_init = bd.gated_scan_bwd(x, back, x, init_state=one, d_final=one)
    assert float((d_init.double() - want).abs().max()) <= off
    for t in (47, 46, 20, 0):
        assert float((dx[:, t].double() - want).abs().max()) <= off and float((da[:, t].double() - want).abs().max()) <= off


@pytest.mark.parametrize("a", [-0.03, -0.06, -0.0624, -0.0625, -0.0626, -0.07])
def test_constant_gates_next_to_the_border(a):
    """A constant gate's error adds up over its memory, 1 / beta tokens: 4 U of the state on the series'
    side, (2 + 2 |a|) U / beta = 36 U next to the border on the other, of tol's 145 U."""
    L, D = 4096, 64
    g = torch.Generator().manual_seed(1)
    x, dy = (torch.rand((1, L, D), generator=g).cuda() + 0.5 for _ in range(2))
    gate = torch.full((1, L, D), a, device="cuda")
    init = torch.full((1, D), 100.0, device="cuda")
    y, final, kept = bd.gated_scan_fwd(x, gate, init_state=init, keep_states=True)
    ey, states = oracle.scan_f64(x, gate, False, init)
    assert rel(y, ey) <= tol(F32, L) and rel(final, states[-1]) <= tol(F32, L)
    ex, ea, _ = oracle.scan_grads_f64(x, gate, False, dy, init)
    dx, da, _ = bd.gated_scan_bwd(x, gate, dy, states=kept)
    assert rel(dx, ex) <= 2 * tol(F32, L) and rel(da, ea) <= 4 * tol(F32, L)
    # the first state's gradient from the last token alone: every one of 512 gates counts
    n = 512
    zero = torch.zeros((1, n, D), device="cuda")
    _, _, d_init = bd.gated_scan_bwd(zero, gate[:, :n].contiguous(), zero, init_state=init, d_final=torch.ones_like(init))
    want = math.exp(n * float(gate[0, 0, 0].double()))
    assert float((d_init.double() / want - 1).abs().max()) <= n * (4 + 2 * abs(a)) * U


# two channels a lane: ragged ends of tokens and channels, short, double and long tiles
PAIRS = [(1, 33, 66), (2, 129, 62), (64, 129, 640), (16, 256, 2050), (3, 600, 66), (4, 700, 2050), (1, 4097, 258)]


@pytest.mark.parametrize("b,L,D", PAIRS)
@pytest.mark.parametrize("a_dtype", [BF, F32])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_every_element_of_bf16_outputs(b, L, D, a_dtype, sigmoid):
    """One rounding of the element (2^-8 of it), and the 32-bit sums' error relative to the largest value
    of the element's channel: tol counts 2 sqrt(L) U, and L roundings of U / 2 at the most have a
    deviation of sqrt(L / 12) U, so that 8 tol are far outside it.  No element can be another one's, or
    none."""
    c = make(b, L, D, sigmoid, BF, a_dtype, seed=L + D + 1)
    y, final, kept = bd.gated_scan_fwd(c["x"], c["a"], sigmoid=sigmoid, init_state=c["init"], keep_states=True)
    ey, states = oracle.scan_f64(c["x"], c["a"], sigmoid, c["init"])
    dx, da, d_init = bd.gated_scan_bwd(c["x"], c["a"], c["dy"], sigmoid=sigmoid, d_final=c["d_final"], states=kept)
    ex, ea, ei = oracle.scan_grads_f64(c["x"], c["a"], sigmoid, c["dy"], c["init"], c["d_final"])
    assert y.dtype == c["x"].dtype and dx.dtype == c["x"].dtype and da.dtype == c["a"].dtype
    slack = 8 * tol(F32, L)
    before = torch.stack(states[:-1], 1)
    a = c["a"].double()
    alpha, beta = (torch.sigmoid(a), torch.sigmoid(-a)) if sigmoid else (torch.exp(a), torch.ones_like(a))
    lam = ex / beta
    top = lambda t: t.abs().amax(1, keepdim=True)
    terms = lam.abs() * alpha * beta * (before.abs() + c["x"].double().abs() if sigmoid else before.abs())
    state = torch.maximum(top(ey), c["init"].double().abs()[:, None])
    for got, want, size, half in ((y, ey, state, 2.0 ** -8), (dx, ex, top(ex) if not sigmoid else top(lam) * beta, 2.0 ** -8),
                                  (da, ea, top(terms), 2.0 ** -8 if a_dtype == BF else U)):
        assert float(((got.double() - want).abs() / (half * want.abs() + slack * size)).max()) <= 1.0
    assert float(((kept.double() - before[:, ::bd.GATED_SCAN_KEEP]).abs() / (slack * state)).max()) <= 1.0
    assert float(((final.double() - states[-1]).abs() / (slack * state[:, 0])).max()) <= 1.0
    assert float(((d_init.double() - ei).abs() / (slack * top(lam)[:, 0].clamp_min(float(c["d_final"].abs().max())))).max()) <= 1.0
