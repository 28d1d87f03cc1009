"""A NaN or an infinity among the inputs of one token of the gated delta rule: the outputs of
earlier tokens, of the same chunk too, and of what else does not depend on it are bit for
bit those without it (MI355X only)."""
import pytest
import torch

from delta_helpers import inputs_of, make
from selective_state_space_ssd_amd import binding as bd

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NAN, INF = float("nan"), float("inf")
# b, L, H, G, P, N: a ragged last chunk, waves that share their rows among 1, 2 and 4, segments
SHAPES = [(1, 150, 4, 2, 32, 32), (1, 130, 4, 2, 64, 64), (2, 100, 2, 1, 48, 128), (1, 1100, 2, 1, 32, 128), (1, 100, 70, 2, 64, 64), (1, 90, 132, 2, 64, 128),
          (1, 80, 2, 1, 32, 256)]


def run(c):
    return bd.gated_delta_fwd(*inputs_of(c), 0.5, init_state=c["init_state"])


@pytest.mark.parametrize("b,L,H,G,P,N", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("token", [0, 1, 17, 37, 63, -1])
@pytest.mark.parametrize("value", [NAN, INF])
def test_a_value_stops_at_its_token(b, L, H, G, P, N, dtype, token, value):
    c = make(b, L, H, G, P, N, dtype, seed=L)
    y0, S0 = run(c)
    t = L // 64 * 64 - 64 + token if token >= 0 else L - 1     # of the last whole chunk, or the last of all
    x = dict(c, v=c["v"].clone())
    x["v"][0, t, 1, 5] = value
    y, S = run(x)
    assert torch.equal(y[:, :t], y0[:, :t])
    others = torch.ones(b, H, P, dtype=torch.bool, device="cuda")
    others[0, 1, 5] = False
    assert torch.equal(S[others], S0[others])
    assert torch.equal(y[:, t:].movedim(1, -1)[others], y0[:, t:].movedim(1, -1)[others])
    assert not torch.isfinite(y[0, t:, 1, 5]).any() and not torch.isfinite(S[0, 1, 5]).any()


@pytest.mark.parametrize("b,L,H,G,P,N", SHAPES[:3])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("token", [0, 18, 37, 50, 63])
@pytest.mark.parametrize("name", ["q", "k", "a", "beta"])
def test_of_keys_queries_and_gates(b, L, H, G, P, N, dtype, token, name):
    c = make(b, L, H, G, P, N, dtype, seed=L)
    y0, S0 = run(c)
    x = dict(c)
    x[name] = c[name].clone()
    x[name][(0, token, 0, 3) if name in "qk" else (0, token, 0)] = NAN
    y, S = run(x)
    heads = range(H // G) if name in "qk" else range(1)        # those that see it
    assert torch.equal(y[:, :token], y0[:, :token])
    rest = [h for h in range(H) if h not in heads]
    assert torch.equal(y[:, :, rest], y0[:, :, rest]) and torch.equal(S[:, rest], S0[:, rest])
    for h in heads:
        assert torch.isnan(y[0, token, h]).all()
        if name == "q":
            assert torch.equal(y[0, token + 1:, h], y0[0, token + 1:, h]) and torch.equal(S[0, h], S0[0, h])
        else:
            assert torch.isnan(y[0, token:, h]).all() and torch.isnan(S[0, h]).all()
