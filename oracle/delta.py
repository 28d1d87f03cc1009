"""The gated delta rule in float64, token by token, and its gradients by automatic
differentiation of those lines (torch, on the CPU or wherever the inputs are).

Shapes as in the library: q, k [b, L, G, N]; v [b, L, H, P]; a, beta [b, L, H]; states
[b, H, P, N].  Test infrastructure; it shares no code with the HIP path.
"""
from __future__ import annotations

import torch


def _f64(x):
    return None if x is None else x.detach().to(torch.float64)


def _recurrence(q, k, v, a, beta, state, scale):
    b, L, H, P = v.shape
    r = H // k.shape[2]
    ys, states = [], [state]
    S = state
    for t in range(L):
        kt = k[:, t].repeat_interleave(r, dim=1)
        qt = q[:, t].repeat_interleave(r, dim=1)
        S = torch.exp(a[:, t])[:, :, None, None] * S
        u = beta[:, t][..., None] * (v[:, t] - (S * kt[:, :, None, :]).sum(-1))
        S = S + u[..., None] * kt[:, :, None, :]
        ys.append(scale * (S * qt[:, :, None, :]).sum(-1))
        states.append(S)
    y = torch.stack(ys, 1) if ys else v.new_zeros(v.shape)
    return y, states


def _start(v, k, init_state):
    if init_state is not None:
        return _f64(init_state)
    b, _, H, P = v.shape
    return torch.zeros(b, H, P, k.shape[3], dtype=torch.float64, device=v.device)


def delta_f64(q, k, v, a, beta, scale, init_state=None):
    """(y, states): states[t] is the state after t tokens, t = 0 .. L."""
    S = _start(v, k, init_state)
    return _recurrence(*(_f64(x) for x in (q, k, v, a, beta)), S, scale)


def delta_grads_f64(q, k, v, a, beta, scale, dy, init_state=None, d_final=None):
    """(dq, dk, dv, da, dbeta, d_init) of sum(dy y) + sum(d_final final_state)."""
    leaves = [_f64(x).requires_grad_() for x in (q, k, v, a, beta)]
    leaves.append(_start(v, k, init_state).requires_grad_())
    with torch.enable_grad():
        y, states = _recurrence(*leaves, scale)
        loss = (_f64(dy) * y).sum()
        if d_final is not None:
            loss = loss + (_f64(d_final) * states[-1]).sum()
        grads = torch.autograd.grad(loss, leaves, allow_unused=True)
    return tuple(torch.zeros_like(x) if g is None else g for x, g in zip(leaves, grads))
