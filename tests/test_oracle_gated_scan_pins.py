"""Pins of the float64 forms of the gated scan, of the dropout's generator and of the 8-bit
norm: facts outside themselves (CPU only)."""
import math

import numpy as np
import pytest
import torch

from oracle import gated_scan, norms


def t64(*v):
    return torch.tensor(v, dtype=torch.float64)


def test_two_tokens_by_hand():
    # h0 = 4; a = ln 1/2, x = 3: h = 5; a = ln 1/5, x = -2: h = -1
    y, s = gated_scan.scan_f64(t64(3, -2).view(1, 2, 1), t64(math.log(0.5), math.log(0.2)).view(1, 2, 1), False, t64(4.0).view(1, 1))
    assert torch.allclose(y.flatten(), t64(5, -1)) and torch.allclose(s[-1].flatten(), t64(-1))
    # a gate of 0 halves both: (4 + 3) / 2 = 3.5, (3.5 - 2) / 2 = 0.75
    y, _ = gated_scan.scan_f64(t64(3, -2).view(1, 2, 1), torch.zeros(1, 2, 1), True, t64(4.0).view(1, 1))
    assert torch.allclose(y.flatten(), t64(3.5, 0.75))


def test_constant_gate_is_a_library_filter():
    from scipy.signal import lfilter
    x = torch.randn(1, 200, 3, generator=torch.Generator().manual_seed(0), dtype=torch.float64)
    y, _ = gated_scan.scan_f64(x, torch.full((1, 200, 3), math.log(0.9), dtype=torch.float64), False)
    assert np.allclose(y.numpy(), lfilter([1.0], [1.0, -0.9], x.numpy(), axis=1), rtol=1e-12, atol=1e-12)


def test_open_and_closed_gates():
    x = torch.randn(2, 9, 4, generator=torch.Generator().manual_seed(1), dtype=torch.float64)
    y, _ = gated_scan.scan_f64(x, torch.zeros_like(x), False)
    assert torch.allclose(y, x.cumsum(1))                     # nothing decays
    y, _ = gated_scan.scan_f64(x, torch.full_like(x, -math.inf), False)
    assert torch.equal(y, x)                                  # everything is forgotten
    y, _ = gated_scan.scan_f64(x, torch.full_like(x, -math.inf), True)
    assert torch.equal(y, x)
    y, s = gated_scan.scan_f64(x, torch.full_like(x, math.inf), True, torch.ones(2, 4))
    assert torch.equal(s[-1], torch.ones(2, 4, dtype=torch.float64))


@pytest.mark.parametrize("sigmoid", [False, True])
def test_gradients_against_differences(sigmoid):
    g = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)
    x, a, init, dy, d_final = r(2, 7, 3), r(2, 7, 3), r(2, 3), r(2, 7, 3), r(2, 3)
    a = a if sigmoid else -a.abs()

    def loss(x, a, init):
        y, s = gated_scan.scan_f64(x, a, sigmoid, init)
        return float((dy * y).sum() + (d_final * s[-1]).sum())

    grads = gated_scan.scan_grads_f64(x, a, sigmoid, dy, init, d_final)
    for i, d in enumerate(grads):
        args = [x, a, init]
        way, h = r(*d.shape), 1e-6
        up, down = (loss(*(args[:i] + [args[i] + s * h * way] + args[i + 1:])) for s in (1, -1))
        assert (up - down) / (2 * h) == pytest.approx(float((d * way).sum()), rel=1e-6, abs=1e-7)


def test_no_tokens():
    x = torch.zeros(2, 0, 3)
    y, s = gated_scan.scan_f64(x, x, False, torch.ones(2, 3))
    assert y.shape == (2, 0, 3) and torch.equal(s[-1], torch.ones(2, 3, dtype=torch.float64))
    dx, da, d_init = gated_scan.scan_grads_f64(x, x, False, x, None, torch.ones(2, 3))
    assert dx.shape == da.shape == (2, 0, 3) and torch.equal(d_init, torch.ones(2, 3, dtype=torch.float64))


def test_generator_against_published_words():
    """The known answers of the generator's authors: counter and key all zeros, all ones, and
    digits of pi."""
    def words(counter, key):
        at = counter[0] | counter[1] << 32
        return [int(w) for w in norms.philox_words(4, key[0] | key[1] << 32, counter[2] | counter[3] << 32, first=4 * at)]

    assert words((0, 0, 0, 0), (0, 0)) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    # the other two by the same rounds in plain integers (their counters lie past any array)
    def plain(c, k):
        for _ in range(10):
            p, q = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
            c = (q >> 32 ^ c[1] ^ k[0], q & 0xFFFFFFFF, p >> 32 ^ c[3] ^ k[1], p & 0xFFFFFFFF)
            k = ((k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF)
        return list(c)

    ones = 0xFFFFFFFF
    assert plain((ones,) * 4, (ones, ones)) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert plain((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0)) == [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]
    seed, offset = 0x1234567890ABCDEF, 0xFEDCBA0987654321
    for at, up in ((0, 0), (1, 0), (77, 0), (5, 9)):
        assert words((at, up, offset & ones, offset >> 32), (seed & ones, seed >> 32)) == plain((at, up, offset & ones, offset >> 32), (seed & ones, seed >> 32))


def test_dropout_keeps_its_share():
    n = 1 << 20
    for p in (0.1, 0.5):
        f = norms.dropout_factor((n,), p, (7, 9))
        # the share that stays is binomial: within six standard deviations
        assert abs(float((f > 0).double().mean()) - (1 - p)) < 6 * math.sqrt(p * (1 - p) / n)
    assert bool((norms.dropout_factor((10,), 0.0, (1, 2)) == 1).all())


def test_scales_of_groups():
    q, s = norms.q8_of(t64(1, -2, 0.5, 0, 0, 0).view(1, 6), 3)
    assert torch.allclose(s, t64(2 / 448, 2.0 ** -126).view(1, 2)) and torch.allclose(q, t64(224, -448, 112, 0, 0, 0).view(1, 6))
