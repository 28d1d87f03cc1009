"""Pins of the float64 forms of the gated delta rule and of the norms: facts outside
themselves (CPU only)."""
import math

import pytest
import torch

from delta_helpers import inputs_of, make
from oracle import delta, norms


def test_one_token_by_hand():
    # S = 2, a = ln(1/2), k = 3, v = 10, beta = 1/2, q = 4, scale = 1/4:
    # S' = 1, u = (10 - 3) / 2 = 3.5, S = 1 + 10.5 = 11.5, y = 11.5
    t = lambda *v: torch.tensor(v, dtype=torch.float64)
    y, s = delta.delta_f64(t(4.0).view(1, 1, 1, 1), t(3.0).view(1, 1, 1, 1), t(10.0).view(1, 1, 1, 1),
                           t(math.log(0.5)).view(1, 1, 1), t(0.5).view(1, 1, 1), 0.25, t(2.0).view(1, 1, 1, 1))
    assert float(y) == pytest.approx(11.5) and float(s[-1]) == pytest.approx(11.5)


def test_orthogonal_keys_are_read_back():
    # without decay and with beta = 1, distinct unit keys hold their values
    n = 8
    k = torch.eye(n).view(1, n, 1, n)
    v = torch.randn(1, n, 1, 5, generator=torch.Generator().manual_seed(0))
    y, s = delta.delta_f64(k, k, v, torch.zeros(1, n, 1), torch.ones(1, n, 1), 1.0)
    assert torch.allclose(y, v.double()) and torch.allclose(s[-1][0, 0], v[0, :, 0].double().T)


def test_a_key_written_twice_holds_the_last_value():
    k = torch.zeros(1, 2, 1, 4)
    k[..., 1] = 1.0
    v = torch.randn(1, 2, 1, 3, generator=torch.Generator().manual_seed(1))
    _, s = delta.delta_f64(k, k, v, torch.zeros(1, 2, 1), torch.ones(1, 2, 1), 1.0)
    assert torch.allclose(s[-1][0, 0, :, 1], v[0, 1, 0].double())


def test_delta_gradients_against_differences():
    c = make(2, 5, 4, 2, 3, 4, torch.float32, seed=2, device="cpu")
    args = [t.double() for t in inputs_of(c)] + [c["init_state"].double()]
    grads = delta.delta_grads_f64(*args[:5], 0.8, c["dy"], args[5], c["d_final"])

    def loss(x):
        y, s = delta.delta_f64(*x[:5], 0.8, x[5])
        return float((c["dy"].double() * y).sum() + (c["d_final"].double() * s[-1]).sum())

    g = torch.Generator().manual_seed(3)
    for i, (x, d) in enumerate(zip(args, grads)):
        way = torch.randn(x.shape, generator=g, dtype=torch.float64)
        h = 1e-5
        up, down = (loss(args[:i] + [x + s * h * way] + args[i + 1:]) for s in (1, -1))
        assert (up - down) / (2 * h) == pytest.approx(float((d * way).sum()), rel=1e-6, abs=1e-7)


@pytest.mark.parametrize("gate_first", [False, True])
def test_norm_gate_gradients_against_differences(gate_first):
    g = torch.Generator().manual_seed(4)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)
    args, dy = [r(3, 6), r(3, 6), r(6)], r(3, 6)
    grads = norms.norm_gate_grads_f64(*args, dy, 3, 1e-5, gate_first)
    for i, (x, d) in enumerate(zip(args, grads)):
        way, h = r(*x.shape), 1e-6
        up, down = (float((dy * norms.norm_gate_f64(*(args[:i] + [x + s * h * way] + args[i + 1:]), 3, 1e-5, gate_first)).sum()) for s in (1, -1))
        assert (up - down) / (2 * h) == pytest.approx(float((d * way).sum()), rel=1e-6, abs=1e-7)


def test_norm_add_gradients_against_differences():
    g = torch.Generator().manual_seed(5)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)
    x, res, w, sc, dy, d_sum = r(3, 6), r(3, 6), r(6), r(6), r(3, 6), r(3, 6)

    def loss(x, res, w, sc):
        total = res + sc * x
        y = total / torch.sqrt((total * total).mean(-1, keepdim=True) + 1e-5) * w
        return float((dy * y).sum() + (d_sum * total).sum())

    dx, dres, dw, dsc = norms.norm_add_grads_f64(x, res + sc * x, w, dy, d_sum, 1e-5, sc)
    args = [x, res, w, sc]
    for i, d in enumerate((dx, dres, dw, dsc)):
        way, h = r(*args[i].shape), 1e-6
        up, down = (loss(*(args[:i] + [args[i] + s * h * way] + args[i + 1:])) for s in (1, -1))
        assert (up - down) / (2 * h) == pytest.approx(float((d * way).sum()), rel=1e-6, abs=1e-7)


def test_a_constant_row_has_norm_one():
    y = norms.norm_gate_f64(torch.full((1, 8), 3.0), None, torch.ones(8), 8, 0.0, False)
    assert torch.allclose(y, torch.ones(1, 8, dtype=torch.float64))
    y, total = norms.norm_add_f64(torch.full((1, 4), 2.0), torch.full((1, 4), 1.0), torch.ones(4), 0.0, torch.full((4,), 0.5))
    assert torch.allclose(total, torch.full((1, 4), 2.0, dtype=torch.float64)) and torch.allclose(y, torch.ones(1, 4, dtype=torch.float64))
