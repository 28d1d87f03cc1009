"""Inputs of the gated delta rule's GPU tests, and the measure of their comparisons."""
import math

import torch

U32 = 2.0 ** -24


def rel(got, want):
    """2-norm of the difference over the 2-norm of ``want`` (the difference's own where
    ``want`` is zero)."""
    got, want = got.double().cpu(), want.double().cpu()
    assert got.shape == want.shape
    if not want.numel():
        return 0.0
    n, d = float(want.norm()), float((got - want).norm())
    return d / n if n else d


def make(b, L, H, G, P, N, dtype, seed=0, init=True, device="cuda"):
    """Unit keys and queries, gates of a softplus step times a rate per head."""
    g = torch.Generator().manual_seed(seed)

    def normal(*s):
        return torch.randn(s, generator=g)

    unit = lambda x: torch.nn.functional.normalize(x, dim=-1)
    rate = torch.exp(torch.rand(H, generator=g) * math.log(16.0))
    c = dict(q=unit(normal(b, L, G, N)).to(dtype), k=unit(normal(b, L, G, N)).to(dtype), v=normal(b, L, H, P).to(dtype),
             a=-rate * torch.nn.functional.softplus(normal(b, L, H) - 4.6).clamp(1e-3, 1e-1), beta=torch.sigmoid(normal(b, L, H)))
    c["init_state"] = 0.1 * normal(b, H, P, N) if init else None
    c["dy"], c["d_final"] = normal(b, L, H, P).to(dtype), normal(b, H, P, N)
    return {n: t if t is None else t.to(device) for n, t in c.items()}


def inputs_of(c):
    return [c[n] for n in ("q", "k", "v", "a", "beta")]


def tol32(L, N):
    """Of a value carried in 32 bits: every token takes sums of N terms and adds a
    rounding to a state that no later token enlarges; the errors are independent."""
    return (16 + 4 * math.sqrt(N) + 2 * math.sqrt(L)) * U32


def tol_out(dtype, L, N, roundings):
    """Of an output of type ``dtype`` behind that many roundings to bf16."""
    if dtype == torch.float32:
        return tol32(L, N)
    return roundings * torch.finfo(dtype).eps / 2 + tol32(L, N)


# b, L, H, G, P, N with so many heads that a wave has 16 rows of the state to itself or
# shares them with one other (the small cases share them among four), blocks whose last
# rows lie past the head, and many chunks (so many that the gradients' sums are split in the
# middle of a head); last, more tiles of 16 rows than the device has SIMDs
MANY = [(1, 70, 132, 1, 64, 64), (1, 70, 40, 1, 208, 64), (1, 70, 70, 2, 64, 128), (1, 70, 18, 2, 240, 128), (1, 70, 132, 2, 64, 128),
        (1, 66, 70, 2, 64, 256), (1, 66, 18, 3, 240, 256), (9, 900, 8, 4, 16, 32), (8, 1000, 3, 1, 80, 32),
        (1, 66, 118, 1, 144, 64), (2, 100, 33, 3, 256, 32), (1, 66, 132, 2, 128, 128)]

# b, L, H, G, P, N of sequences long enough for their few heads to be cut into segments: a
# ragged last segment, blocks that end in the middle of a head's rows, every state width
CUT = [(1, 64 * 16, 1, 1, 16, 32), (1, 64 * 40 - 63, 2, 1, 48, 64), (2, 64 * 30 + 1, 1, 1, 80, 128), (1, 2500, 3, 1, 32, 128), (1, 1600, 1, 1, 64, 256),
       (1, 64 * 100, 1, 1, 16, 64)]
