"""The gated scan over shapes that reach each of its kernels' tiles and each way of finding the
entering state: few blocks and many, one and two channels a lane, sequences of more blocks
than are looked back over, offsets past 2^31 elements (MI355X only).  Tolerances:
scan_helpers.tol."""
import math

import pytest
import torch

from oracle import gated_scan as oracle
from scan_helpers import check_bwd, check_fwd, make, rel, tol
from selective_state_space_ssd_amd import binding as bd

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

# b, L, D: more blocks than CUs with two channels a lane and with one (odd D), ragged in tokens
# and channels; the last length of a short tile and lengths of a double one; long chains of few blocks
TILES = [(4, 700, 2050), (3, 600, 2047), (64, 128, 640), (64, 129, 640), (2, 129, 67), (4, 200, 640), (16, 256, 2050), (1, 4096, 258), (1, 4097, 258), (1, 9000, 6), (2, 9217, 1)]


@pytest.mark.parametrize("b,L,D", TILES)
@pytest.mark.parametrize("dtype,a_dtype", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_tiles(b, L, D, dtype, a_dtype, sigmoid):
    c = make(b, L, D, sigmoid, dtype, a_dtype, seed=L + D, init=L % 2 == 1)
    y, final, kept = bd.gated_scan_fwd(c["x"], c["a"], sigmoid=sigmoid, init_state=c["init"], keep_states=True)
    want = oracle.scan_f64(c["x"], c["a"], sigmoid, c["init"])
    check_fwd(c, sigmoid, (y, final), want)
    assert rel(kept, torch.stack(want[1][:-1:bd.GATED_SCAN_KEEP], 1)) <= tol(F32, L)
    got = bd.gated_scan_bwd(c["x"], c["a"], c["dy"], sigmoid=sigmoid, init_state=c["init"], d_final=c["d_final"], states=kept)
    check_bwd(c, sigmoid, got, oracle.scan_grads_f64(c["x"], c["a"], sigmoid, c["dy"], c["init"], c["d_final"]), want[1])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [1, 64])
def test_more_blocks_than_are_looked_back_over(dtype, D):
    """60001 tokens that hardly forget: the state at the end is made by all of them.  (Forward
    alone in float64: the states of the reference take 60001 x D x 8 bytes.)"""
    L = 60001
    g = torch.Generator().manual_seed(3)
    x = torch.randn((1, L, D), generator=g).to(dtype).cuda()
    a = (-1e-5 * torch.rand((1, L, D), generator=g)).cuda()
    y, final = bd.gated_scan_fwd(x, a, init_state=torch.full((1, D), 50.0, device="cuda"))
    ey, states = oracle.scan_f64(x, a, False, torch.full((1, D), 50.0, device="cuda"))
    assert rel(y, ey) <= tol(dtype, L) and rel(final, states[-1]) <= tol(F32, L)
    # the gradient of the first token's state from the last token's alone
    dy = torch.zeros_like(x)
    _, _, d_init = bd.gated_scan_bwd(x, a, dy, d_final=torch.ones((1, D), device="cuda"))
    assert rel(d_init, a.double().sum(1).exp()) <= tol(F32, L)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_long_chain_repeats_and_holds_a_nan_back(sigmoid):
    c = make(1, 30000, 34, sigmoid, BF, F32, seed=9)
    run = lambda: bd.gated_scan_fwd(c["x"], c["a"], sigmoid=sigmoid, init_state=c["init"]) + bd.gated_scan_bwd(
        c["x"], c["a"], c["dy"], sigmoid=sigmoid, init_state=c["init"], d_final=c["d_final"])
    first = run()
    for _ in range(3):
        assert all(torch.equal(s, t) for s, t in zip(first, run()))
    c["x"][0, 20000, 7] = float("nan")
    y = bd.gated_scan_fwd(c["x"], c["a"], sigmoid=sigmoid, init_state=c["init"])[0]
    others = [i for i in range(34) if i != 7]
    assert torch.equal(y[:, :20000], first[0][:, :20000]) and torch.equal(y[..., others], first[0][..., others])
    assert bool(y[0, 20000:, 7].isnan().all())


def test_offsets_past_31_bits():
    """2^20 + 5 tokens of 2056 channels, 4.3 GB an array: the gates are closed 90 tokens before
    the end, so that what comes out there is the last tokens' own."""
    L, D, n = (1 << 20) + 5, 2056, 90
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.empty((1, L, D), dtype=BF, device="cuda").normal_(generator=g)
    a = torch.full((1, L, D), -0.01, dtype=BF, device="cuda")
    a[:, L - n] = -math.inf
    y, final, kept = bd.gated_scan_fwd(x, a, keep_states=True)
    tail = [t[:, L - n:].contiguous() for t in (x, a)]
    ey, states = oracle.scan_f64(*tail, False)
    assert rel(y[:, L - n:], ey) <= tol(BF, n) and rel(final, states[-1]) <= tol(F32, n)
    ey, _ = oracle.scan_f64(x[:, :n].contiguous(), a[:, :n].contiguous(), False)
    assert rel(y[:, :n], ey) <= tol(BF, n)
    del y
    # gradients of the last tokens, and none behind the closed gate
    dy = torch.zeros_like(x)
    dy[:, L - 60:] = 1.0
    dx, da, _ = bd.gated_scan_bwd(x, a, dy, states=kept)
    ex, ea, _ = oracle.scan_grads_f64(*tail, False, dy[:, L - n:].contiguous())
    assert rel(dx[:, L - n:], ex) <= 2 * tol(BF, n) and rel(da[:, L - n:], ea) <= 2 * tol(BF, n)
    assert float(dx[:, L - n - 500:L - n].abs().max()) == 0.0 and float(da[:, L - n - 500:L - n].abs().max()) == 0.0
