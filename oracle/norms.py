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


def philox_words(n, seed, offset, first=0):
    """Words first .. first + n - 1 (first a multiple of 4) of Philox4x32-10: word i is word
    i mod 4 of the counter (i / 4, offset) under the key seed.  numpy, on the CPU."""
    import numpy as np
    u = np.uint64
    mask, i = u(0xFFFFFFFF), np.arange((n + 3) // 4, dtype=np.uint64) + u(first // 4)
    seed, offset = int(seed) % (1 << 64), int(offset) % (1 << 64)
    c0, c1 = i & mask, i >> u(32)
    c2, c3 = np.full_like(i, offset & 0xFFFFFFFF), np.full_like(i, offset >> 32)
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        p, q = u(0xD2511F53) * c0, u(0xCD9E8D57) * c2
        c0, c1, c2, c3 = (q >> u(32)) ^ c1 ^ u(k0), q & mask, (p >> u(32)) ^ c3 ^ u(k1), p & mask
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack([c0, c1, c2, c3], 1).reshape(-1)[:n].astype(np.uint32)


def dropout_factor(shape, p, rng):
    """0 or 1 / (1 - p) per element (float64): what x is multiplied by.  p as 32 bits hold it."""
    import numpy as np
    n, p = int(np.prod(shape)), float(np.float32(p))
    stays = philox_words(n, int(rng[0]), int(rng[1])) >= np.uint32(int(p * 4294967296.0))
    return torch.from_numpy(stays).reshape(shape).to(torch.float64) / (1.0 - p)


def q8_of(y, group):
    """(y / scale, scale) per group of channels, before the rounding to e4m3."""
    g = y.reshape(*y.shape[:-1], y.shape[-1] // group, group)
    scale = torch.clamp_min(g.abs().amax(-1) / 448.0, 2.0 ** -126)
    return (g / scale[..., None]).reshape(y.shape), scale
