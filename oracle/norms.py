"""The norms around a block in float64 (torch), and their gradients by automatic
differentiation.  Test infrastructure; it shares no code with the HIP path."""
from __future__ import annotations

import torch


def _f64(x):
    return None if x is None else x.detach().to(torch.float64)


def _normed(u, group, eps):
    shape = u.shape
    u = u.reshape(*shape[:-1], shape[-1] // group, group)
    return (u / torch.sqrt((u * u).mean(-1, keepdim=True) + eps)).reshape(shape)


def _gate(x, z, w, group, eps, gate_first):
    act = 1.0 if z is None else z * torch.sigmoid(z)
    return _normed(x * act, group, eps) * w if gate_first else _normed(x, group, eps) * w * act


def norm_gate_f64(x, z, w, group, eps, gate_first):
    return _gate(_f64(x), _f64(z), _f64(w), group, eps, gate_first)


def norm_gate_grads_f64(x, z, w, dy, group, eps, gate_first):
    """(dx, dz, dw); dz None without z."""
    leaves = [t if t is None else _f64(t).requires_grad_() for t in (x, z, w)]
    with torch.enable_grad():
        y = _gate(*leaves, group, eps, gate_first)
        grads = iter(torch.autograd.grad((_f64(dy) * y).sum(), [t for t in leaves if t is not None]))
    return tuple(None if t is None else next(grads) for t in leaves)


def norm_add_f64(x, residual, w, eps, scale=None):
    """(y, sum); the norm sees the sum as it is stored, in the residual's type."""
    total = _f64(residual) + (_f64(x) if scale is None else _f64(scale) * _f64(x))
    held = total.to(torch.float32).to(residual.dtype).to(torch.float64)
    return _normed(held, held.shape[-1], eps) * _f64(w), total


def norm_add_grads_f64(x, total, w, dy, d_sum, eps, scale=None):
    """(dx, d_residual, dw, d_scale) with the sum as stored; d_scale None without scale."""
    s, w64 = _f64(total).requires_grad_(), _f64(w).requires_grad_()
    with torch.enable_grad():
        loss = (_f64(dy) * _normed(s, s.shape[-1], eps) * w64).sum()
        if d_sum is not None:
            loss = loss + (_f64(d_sum) * s).sum()
        ds, dw = torch.autograd.grad(loss, (s, w64))
    if scale is None:
        return ds, ds, dw, None
    return ds * _f64(scale), ds, dw, (ds * _f64(x)).reshape(-1, s.shape[-1]).sum(0)
