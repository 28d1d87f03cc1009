"""The forward norms over more segments than one dimension of a launch can count threads for:
2^28 and some, 16 to a block of 256 (MI355X only).  Tolerances as in test_gpu_norms."""
import pytest
import torch

from selective_state_space_ssd_amd import binding as bd

pytestmark = pytest.mark.gpu
EPS = 1e-5
ROWS, PIECE = (1 << 24) + 3, 1 << 21


def test_gated_norm_of_single_channels():
    D = 16
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((ROWS, D), generator=g, device="cuda", dtype=torch.bfloat16)
    w = torch.rand(D, generator=g, device="cuda") + 0.5
    y = torch.full((ROWS + 1, D), 7.0, device="cuda", dtype=torch.bfloat16)
    bd.ssd_norm_gate_fwd(x, None, w, y[:ROWS], 1, EPS, False)
    for at in range(0, ROWS, PIECE):
        u = x[at:at + PIECE].double()
        want = u / torch.sqrt(u * u + EPS) * w.double()
        err = (y[at:min(at + PIECE, ROWS)].double() - want).abs()
        assert bool((err <= (2.0 ** -8 + 16 * 2.0 ** -24) * want.abs()).all()), at
    assert bool((y[ROWS] == 7.0).all())


def test_residual_norm_of_single_channels():
    rows = ROWS * 16
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((rows, 1), generator=g, device="cuda", dtype=torch.bfloat16)
    res = torch.randn((rows, 1), generator=g, device="cuda", dtype=torch.bfloat16)
    w = torch.tensor([1.25], device="cuda")
    y, total = bd.norm_add_fwd(x, res, w, EPS)
    for at in range(0, rows, 16 * PIECE):
        here = slice(at, at + 16 * PIECE)
        s = x[here].double() + res[here].double()
        assert bool(((total[here].double() - s).abs() <= (2.0 ** -8 + 2.0 ** -24) * s.abs()).all()), at
        held = total[here].double()
        want = held / torch.sqrt(held * held + EPS) * 1.25
        assert bool(((y[here].double() - want).abs() <= (2.0 ** -8 + 16 * 2.0 ** -24) * want.abs()).all()), at
