"""The gated scan in float64, token by token, and its gradients by automatic differentiation
of those lines (torch, on the CPU or wherever the inputs are).

Shapes as in the library: x, a [b, L, D]; states [b, D].  Test infrastructure; it shares no
code with the HIP path.
"""
from __future__ import annotations

import torch


def _f64(x):
    return None if x is None else x.detach().to(torch.float64)


def _recurrence(x, a, h, sigmoid):
    states = [h]
    alpha = torch.sigmoid(a) if sigmoid else torch.exp(a)
    u = torch.sigmoid(-a) * x if sigmoid else x
    for t in range(x.shape[1]):
        h = alpha[:, t] * h + u[:, t]
        states.append(h)
    return states


def _start(x, init_state):
    b, _, D = x.shape
    return torch.zeros(b, D, dtype=torch.float64, device=x.device) if init_state is None else _f64(init_state)


def scan_f64(x, a, sigmoid, init_state=None):
    """(y, states): states[t] is the state after t tokens, t = 0 .. L."""
    states = _recurrence(_f64(x), _f64(a), _start(x, init_state), sigmoid)
    y = torch.stack(states[1:], 1) if x.shape[1] else _f64(x)
    return y, states


def scan_grads_f64(x, a, sigmoid, dy, init_state=None, d_final=None):
    """(dx, da, d_init) of sum(dy y) + sum(d_final final_state)."""
    leaves = [_f64(t).requires_grad_() for t in (x, a)] + [_start(x, init_state).requires_grad_()]
    with torch.enable_grad():
        states = _recurrence(*leaves, sigmoid)
        loss = sum((_f64(dy)[:, t] * h).sum() for t, h in enumerate(states[1:])) + 0.0 * leaves[2].sum()
        if d_final is not None:
            loss = loss + (_f64(d_final) * states[-1]).sum()
        grads = torch.autograd.grad(loss, leaves, allow_unused=True)
    return tuple(torch.zeros_like(x) if g is None else g for x, g in zip(leaves, grads))
