"""A residual block around the gated scan, the operators run together as a model uses them
(MI355X only):

  training   residual sum with dropout and norm -> projections -> gated scan -> gated norm, and
             back through all of them by the library's gradients;
  serving    residual sum and norm in 8 bits -> projections -> gated scan, a prompt at once and
             then token by token.

The projections are torch products in fp32.  Training is compared with float64 automatic
differentiation of the block's formulas: five operators and three products in a row, forward
and backward, each of them within (16 + 2 sqrt(n)) 2^-24 of its terms with n <= 150, are
within 16 x 41 x 2^-24 < 4e-5 of the result; the gradients are differences of terms a few times
their size, 4 times that.
"""
import pytest
import torch

from oracle import norms
from scan_helpers import rel
from selective_state_space_ssd_amd import binding as bd

pytestmark = pytest.mark.gpu
EPS, TOL = 1e-5, 4e-5


def params(D, E, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)
    return {n: t.cuda() for n, t in dict(w=1 + 0.2 * r(D), ls=0.5 + 0.1 * r(D), Wa=r(D, E) / D ** 0.5, Wu=r(D, E) / D ** 0.5,
                                         Wz=r(D, E) / D ** 0.5, w2=1 + 0.2 * r(E)).items()}


def inputs(b, L, D, E, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g).cuda()
    return r(b, L, D), 2 * r(b, L, D), r(b, E), r(b, L, E), r(b, L, D), r(b, E)


def block_f64(x, residual, h0, p, factor, group):
    total = residual + p["ls"] * x * factor
    y = total / torch.sqrt((total * total).mean(-1, keepdim=True) + EPS) * p["w"]
    a, u, z = y @ p["Wa"], y @ p["Wu"], y @ p["Wz"]
    h, hs = h0, []
    for t in range(x.shape[1]):
        h = torch.sigmoid(a[:, t]) * h + torch.sigmoid(-a[:, t]) * u[:, t]
        hs.append(h)
    k = torch.stack(hs, 1)
    n = k.reshape(*k.shape[:-1], -1, group)
    n = (n / torch.sqrt((n * n).mean(-1, keepdim=True) + EPS)).reshape(k.shape)
    return n * p["w2"] * z * torch.sigmoid(z), total, h


@pytest.mark.parametrize("b,L,D,E,group", [(2, 150, 96, 64, 16), (1, 70, 33, 24, 24)])
def test_training_step(b, L, D, E, group):
    p = params(D, E, 1)
    x, residual, h0, go, gs, gh = inputs(b, L, D, E, 2)
    rng, prob = torch.tensor([11, 12], device="cuda"), 0.2
    y, total = bd.norm_add_drop_fwd(x, residual, p["w"], EPS, prob, rng, scale=p["ls"])
    a, u, z = y @ p["Wa"], y @ p["Wu"], y @ p["Wz"]
    h, final, kept = bd.gated_scan_fwd(u, a, sigmoid=True, init_state=h0, keep_states=True)
    out = bd.norm_gate_fwd(h, z, p["w2"], group, EPS)
    dh, dz, dw2 = bd.norm_gate_bwd(h, z, p["w2"], go, group, EPS)
    du, da, dh0 = bd.gated_scan_bwd(u, a, dh, sigmoid=True, init_state=h0, d_final=gh, states=kept)
    flat = lambda t: t.reshape(-1, t.shape[-1])
    dWa, dWu, dWz = (flat(y).T.contiguous() @ flat(d) for d in (da, du, dz))
    dy = da @ p["Wa"].T.contiguous() + du @ p["Wu"].T.contiguous() + dz @ p["Wz"].T.contiguous()
    dx, dres, dw, dls = bd.norm_add_drop_bwd(x, total, p["w"], dy, gs, EPS, prob, rng, scale=p["ls"])

    factor = norms.dropout_factor((b, L, D), prob, (11, 12)).cuda()
    leaves = {n: t.double().requires_grad_() for n, t in dict(p, x=x, residual=residual, h0=h0).items()}
    want = block_f64(leaves["x"], leaves["residual"], leaves["h0"], leaves, factor, group)
    for got, e in zip((out, total, final), want):
        assert rel(got, e.detach()) <= TOL
    loss = sum((g.double() * e).sum() for g, e in zip((go, gs, gh), want))
    names = ["x", "residual", "h0", "w", "ls", "Wa", "Wu", "Wz", "w2"]
    grads = torch.autograd.grad(loss, [leaves[n] for n in names])
    for name, got, e in zip(names, (dx, dres, dh0, dw, dls, dWa, dWu, dWz, dw2), grads):
        assert rel(got, e) <= 4 * TOL, name


def test_serving_prompt_and_tokens():
    """Rows do not see each other but through the state: the tokens that are decoded one by one
    are those of the whole sequence, up to the products' order of summation (fp32, D = 128
    terms, and a gate and a state behind it)."""
    b, L, D, E = 3, 90, 128, 64
    p = params(D, E, 3)
    x, residual, h0, *_ = inputs(b, L, D, E, 4)

    def inner(xs, rs):
        q, scales, total = bd.norm_add_q8_fwd(xs, rs, p["w"], EPS, group=32, scale=p["ls"])
        y = (q.float().reshape(*q.shape[:-1], -1, 32) * scales[..., None]).reshape(q.shape)
        return y @ p["Wa"], y @ p["Wu"], total

    a, u, total = inner(x, residual)
    whole, last = bd.gated_scan_fwd(u, a, sigmoid=True, init_state=h0)
    n = 80
    cut = lambda t, lo, hi: t[:, lo:hi].contiguous()
    a0, u0, _ = inner(cut(x, 0, n), cut(residual, 0, n))
    _, state = bd.gated_scan_fwd(u0, a0, sigmoid=True, init_state=h0)
    for t in range(n, L):
        at, ut, tt = inner(cut(x, t, t + 1), cut(residual, t, t + 1))
        assert torch.equal(tt, cut(total, t, t + 1))
        y, state = bd.gated_scan_step(state, ut, at, sigmoid=True)
        assert rel(y, cut(whole, t, t + 1)) <= TOL
    assert rel(state, last) <= TOL
