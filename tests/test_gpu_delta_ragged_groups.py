"""The gated delta rule with many chunks and groups whose heads do not divide into the four
that a block of the chunks' preparation takes: the last block of a group has fewer, or all of
its blocks have three (MI355X only)."""
import pytest
import torch

from delta_helpers import inputs_of, make, rel, tol32, tol_out
from oracle import delta
from selective_state_space_ssd_amd import binding as bd

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
# b, L, H, G, P, N: b x 5 chunks x G x ceil(H / G / 4) blocks, 512 and more
GROUPS = [(110, 257, 3, 1, 16, 32), (64, 257, 5, 1, 16, 32), (52, 257, 6, 1, 16, 64), (30, 257, 14, 2, 16, 32), (52, 257, 9, 1, 32, 32)]


@pytest.mark.parametrize("b,L,H,G,P,N", GROUPS)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_outputs_and_gradients(b, L, H, G, P, N, dtype):
    c = make(b, L, H, G, P, N, dtype, seed=H)
    x = {n: t.cpu() for n, t in c.items()}
    y, S = bd.gated_delta_fwd(*inputs_of(c), N ** -0.5, init_state=c["init_state"])
    ey, es = delta.delta_f64(*inputs_of(x), N ** -0.5, x["init_state"])
    got = bd.gated_delta_bwd(*inputs_of(c), N ** -0.5, c["dy"], init_state=c["init_state"], d_final=c["d_final"])
    want = delta.delta_grads_f64(*inputs_of(x), N ** -0.5, x["dy"], x["init_state"], x["d_final"])
    for h in range(H):          # head by head: an error in one is not hidden by the others
        assert rel(y[:, :, h], ey[:, :, h]) <= tol_out(dtype, L, N, 1)
        assert rel(S[:, h], es[-1][:, h]) <= tol32(L, N)
        assert rel(got[2][:, :, h], want[2][:, :, h]) <= tol_out(dtype, L, N, 1) + tol32(L, N)
        for i in (3, 4):
            assert rel(got[i][:, :, h], want[i][:, :, h]) <= 2 * tol32(L, N)
        assert rel(got[5][:, h], want[5][:, h]) <= 2 * tol32(L, N)
    for g in range(G):
        for i in (0, 1):
            assert rel(got[i][:, :, g], want[i][:, :, g]) <= tol_out(dtype, L, N, 1) + tol32(L, N)
