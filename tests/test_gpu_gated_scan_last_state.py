"""The state after the last token is that token's output, an infinite one too, wherever in a
tile the sequence ends (MI355X only)."""
import pytest
import torch

from scan_helpers import make
from selective_state_space_ssd_amd import binding as bd

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("L", [1, 2, 5, 15, 16, 17, 31, 33, 64, 77])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_an_infinite_state(L, sigmoid):
    """alpha between 0.268 and 0.5, finite values: a state of infinity stays one.  (The decays that
    it meets multiplied together are those of the 64 tokens before the last wave's, 2^-122 at the
    least: no 0, which would make it a NaN.)"""
    c = make(2, L, 70, sigmoid, F32, F32, seed=L)
    c["a"].clamp_(-1.0, -0.7)
    if not sigmoid:
        c["a"].fill_(-0.7)
    c["init"][0, ::3] = float("inf")
    c["init"][1, 1::3] = -float("inf")
    y, final = bd.gated_scan_fwd(c["x"], c["a"], sigmoid=sigmoid, init_state=c["init"])
    assert torch.equal(final, y[:, -1])
    assert torch.equal(final.isinf(), c["init"].isinf())
    inf = c["init"].isinf()
    assert torch.equal(final[inf], c["init"][inf])
    ys, state = bd.gated_scan_step(c["init"], c["x"][:, :16].contiguous(), c["a"][:, :16].contiguous(), sigmoid=sigmoid)
    assert torch.equal(state[inf], c["init"][inf])


@pytest.mark.parametrize("L", [1, 31, 33, 300, 700, 1025])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_a_finite_state(L, sigmoid):
    c = make(2, L, 66, sigmoid, F32, F32, seed=L)
    y, final = bd.gated_scan_fwd(c["x"], c["a"], sigmoid=sigmoid, init_state=c["init"])
    assert torch.equal(final, y[:, -1])
    c["x"], c["a"] = c["x"].to(BF), c["a"].to(BF)
    y, final = bd.gated_scan_fwd(c["x"], c["a"], sigmoid=sigmoid, init_state=c["init"])
    assert torch.equal(final.to(BF), y[:, -1])
