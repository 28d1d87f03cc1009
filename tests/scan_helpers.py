"""Inputs of the gated scan's GPU tests, and the measures of their comparisons."""
import math

import torch

U = 2.0 ** -24


def rel(got, want):
    """2-norm of the difference over the 2-norm of ``want`` (the difference's own where
    ``want`` is zero)."""
    got, want = got.double().cpu(), want.double().cpu()
    assert got.shape == want.shape
    if not want.numel():
        return 0.0
    n, d = float(want.norm()), float((got - want).norm())
    return d / n if n else d


def make(b, L, D, sigmoid, dtype, a_dtype, seed=0, init=True):
    """Gates from short memories to long ones, per channel."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)
    if sigmoid:
        a = r(b, L, D) + 6.0 * torch.rand(D, generator=g)
    else:
        a = -torch.nn.functional.softplus(r(b, L, D) - 4.6).clamp(1e-4, 1e-1) * torch.exp(4.0 * torch.rand(D, generator=g))
    c = dict(x=r(b, L, D).to(dtype), a=a.to(a_dtype), init=r(b, D) if init else None, dy=r(b, L, D).to(dtype), d_final=r(b, D))
    return {n: None if t is None else t.cuda() for n, t in c.items()}


def tol(dtype, L):
    """Of a state's trace: one rounding of the output, the gate's few units and, at the worst,
    one rounding of the state a token, independent of each other and none of them enlarged by
    a later token; decays over many tokens are products of as many factors."""
    return (torch.finfo(dtype).eps / 2 if dtype != torch.float32 else U) + (16 + 2 * math.sqrt(L)) * U


def check_fwd(c, sigmoid, got, want):
    """got (y, final) against want (y, states)."""
    L = c["x"].shape[1]
    assert got[0].dtype == c["x"].dtype and got[1].dtype == torch.float32
    assert rel(got[0], want[0]) <= tol(c["x"].dtype, L)
    assert rel(got[1], want[1][-1]) <= tol(torch.float32, L)


def check_bwd(c, sigmoid, got, want, states):
    """got (dx, da, d_init) against want, with the float64 states before each token.  da is a
    product with the state before the token, and behind a gate with its distance from x: its
    error is taken against the terms' size."""
    L, x = c["x"].shape[1], c["x"].double()
    dx, da, d_init = got
    assert dx.dtype == x.dtype or dx.dtype == c["x"].dtype
    assert da.dtype == c["a"].dtype
    assert rel(dx, want[0]) <= 2 * tol(dx.dtype, L)
    if L:
        before = torch.stack(states[:-1], 1)
        a = c["a"].double()
        alpha = torch.sigmoid(a) if sigmoid else torch.exp(a)
        # lambda: dx, with beta taken out again behind a gate; where beta is 0 so is da
        beta = torch.sigmoid(-a)
        lam = torch.where(beta > 0, want[0] / beta, 0.0) if sigmoid else want[0]
        terms = (lam * alpha * (beta * (before.abs() + x.abs()) if sigmoid else before)).norm()
        assert float((da.double() - want[1]).norm()) <= torch.finfo(da.dtype).eps / 2 * float(want[1].norm()) + 4 * tol(torch.float32, L) * float(terms)
    assert rel(d_init, want[2]) <= 2 * tol(torch.float32, L)
