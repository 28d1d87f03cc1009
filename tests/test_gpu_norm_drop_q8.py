"""The residual norm with dropout and with its output in 8 bits against their float64 forms
(MI355X only).

Tolerances as in test_gpu_norms: one rounding of the output plus (16 + 2 sqrt(n)) 2^-24 of
the sums, and for parameters' gradients 2 sqrt(rows) 2^-24 more.  The mask has to be the
generator's, element by element.  e4m3: half a step is 2^-4 of a normal value and 2^-10 (half
the least subnormal 2^-9) below 2^-6; the 32-bit value that is rounded may lie the sums'
tolerance off.
"""
import pytest
import torch

from oracle import norms
from selective_state_space_ssd_amd import binding as bd
from test_gpu_norms import BF, EPS, F32, U, draw, out_tol, par_tol, rel

pytestmark = pytest.mark.gpu

# rows, D: single channels, odd lengths, the last length of a team and one beyond, no team
SHAPES = [(1, 1), (3, 7), (5, 40), (2, 63), (17, 128), (4, 512), (3, 264), (2, 520), (7, 1032), (2, 2056), (2, 5120), (1, 8200), (2, 2047), (3, 2051),
          (2, 12296), (1, 15001), (2100, 16), (600, 24)]
RNG = [(0, 0), (123456789012345678, 42), (-1, -7)]


def state(seed, offset):
    return torch.tensor([seed, offset], dtype=torch.int64, device="cuda")


@pytest.mark.parametrize("rows,D", SHAPES)
@pytest.mark.parametrize("dtype,res", [(BF, F32), (BF, BF), (F32, F32)])
@pytest.mark.parametrize("scaled", [False, True])
def test_dropout_and_gradients(rows, D, dtype, res, scaled):
    x, dy = draw((rows, D), dtype, 1), draw((rows, D), dtype, 3)
    residual, d_sum = draw((rows, D), res, 2, 2.0), draw((rows, D), res, 5)
    w = draw((D,), F32, 4, 0.2, 1.0)
    scale = draw((D,), F32, 6, 0.1, 0.5) if scaled else None
    p, rng = (0.1, 0.3, 0.5)[D % 3], RNG[rows % 3]
    y, total = bd.norm_add_drop_fwd(x, residual, w, EPS, p, state(*rng), scale=scale)
    factor = norms.dropout_factor((rows, D), p, rng).cuda()
    ey, etotal = norms.norm_add_f64(x.double() * factor, residual, w, EPS, scale)
    assert total.dtype == res and y.dtype == dtype
    # an element that is dropped leaves the residual as it was, to the bit
    assert torch.equal(total[factor == 0], residual[factor == 0])
    assert rel(total, etotal) <= torch.finfo(res).eps / 2 + 6 * U
    assert rel(y, ey) <= out_tol(dtype, D) + (6 * U if res == F32 else torch.finfo(res).eps)
    dx, dres, dw, dscale = bd.norm_add_drop_bwd(x, total, w, dy, d_sum, EPS, p, state(*rng), scale=scale)
    ex, eres, ew, escale = norms.norm_add_grads_f64(x.double() * factor, total, w, dy, d_sum, EPS, scale)
    assert bool((dx[factor == 0] == 0).all())
    assert rel(dx, ex * factor) <= 2 * out_tol(dtype, D) and rel(dres, eres) <= 2 * out_tol(res, D)
    assert rel(dw, ew) <= par_tol(D, rows)
    if scaled:
        assert rel(dscale, escale) <= 2 * par_tol(D, rows)
    else:
        assert dscale is None


@pytest.mark.parametrize("D", [96, 95, 15001])
def test_mask_is_the_generators(D):
    """Ones on zeros: the sum is the mask itself.  Rows apart from each other, every word of
    a counter, a counter's both halves of seed and offset."""
    one = torch.ones((4, D), device="cuda")
    for rng in RNG + [(1 << 40, 1 << 50)]:
        for p in (0.0, 0.25, 0.999):
            _, total = bd.norm_add_drop_fwd(one, torch.zeros_like(one), torch.ones(D, device="cuda"), EPS, p, state(*rng))
            want = norms.dropout_factor((4, D), p, rng)
            assert torch.equal(total.cpu() != 0, want != 0)
            assert rel(total.cpu(), want) <= 2 * U


def test_nothing_of_a_dropped_element_is_seen():
    x, residual, w = draw((40, 264), BF, 1), draw((40, 264), F32, 2), draw((264,), F32, 3, 0.2, 1.0)
    scale, dy = draw((264,), F32, 6, 0.1, 0.5), draw((40, 264), BF, 4)
    rng = (5, 6)
    dropped = norms.dropout_factor((40, 264), 0.4, rng).cuda() == 0
    y0, s0 = bd.norm_add_drop_fwd(x, residual, w, EPS, 0.4, state(*rng), scale=scale)
    g0 = bd.norm_add_drop_bwd(x, s0, w, dy, None, EPS, 0.4, state(*rng), scale=scale)
    for bad in (float("nan"), float("inf"), torch.finfo(BF).min):
        x[dropped] = bad
        y, s = bd.norm_add_drop_fwd(x, residual, w, EPS, 0.4, state(*rng), scale=scale)
        assert torch.equal(y, y0) and torch.equal(s, s0)
        g = bd.norm_add_drop_bwd(x, s, w, dy, None, EPS, 0.4, state(*rng), scale=scale)
        assert all(torch.equal(a, b) for a, b in zip(g, g0))


def test_without_dropout_it_is_the_plain_form():
    x, residual, w, dy = draw((9, 520), BF, 1), draw((9, 520), F32, 2), draw((520,), F32, 3, 0.2, 1.0), draw((9, 520), BF, 4)
    assert all(torch.equal(s, t) for s, t in zip(bd.norm_add_drop_fwd(x, residual, w, EPS, 0.0, state(1, 2)), bd.norm_add_fwd(x, residual, w, EPS)))
    got = bd.norm_add_drop_bwd(None, residual, w, dy, None, EPS, 0.0, state(1, 2))
    want = bd.norm_add_bwd(None, residual, w, dy, None, EPS)
    assert all(torch.equal(s, t) for s, t in zip(got[:3], want[:3])) and got[3] is None


def test_dropout_in_place_and_without_rows():
    x, residual, w = draw((9, 320), BF, 1), draw((9, 320), F32, 2), draw((320,), F32, 3, 0.2, 1.0)
    y0, s0 = bd.norm_add_drop_fwd(x, residual, w, EPS, 0.2, state(3, 4))
    y = torch.empty_like(x)
    bd.ssd_norm_add_drop_fwd(x, residual, None, w, state(3, 4), residual, y, EPS, 0.2)
    assert torch.equal(y, y0) and torch.equal(residual, s0)
    e = torch.empty((0, 320), dtype=BF, device="cuda")
    assert bd.norm_add_drop_fwd(e, e, w, EPS, 0.2, state(3, 4))[0].shape == (0, 320)
    _, _, dw, ds = bd.norm_add_drop_bwd(e, e, w, e, None, EPS, 0.2, state(3, 4), scale=w)
    assert float(dw.abs().max()) == 0.0 and float(ds.abs().max()) == 0.0


def test_captured_steps_draw_new_masks():
    """A captured step reads the generator's state when it is replayed."""
    x, residual, w = torch.ones((64, 256), device="cuda"), torch.zeros((64, 256), device="cuda"), torch.ones(256, device="cuda")
    rng, y, total = state(11, 0), torch.empty((64, 256), device="cuda"), torch.empty((64, 256), device="cuda")

    def step():
        bd.ssd_norm_add_drop_fwd(x, residual, None, w, rng, total, y, EPS, 0.5)
        rng[1:].add_(1)

    step()
    rng[1] = 0
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(4):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(total.cpu() != 0, norms.dropout_factor((64, 256), 0.5, (11, k)) != 0)


# ------------------------------------------------------------------------- 8 bits
# rows, D, group: one scale a row; groups within a lane's vector, of 2^k lanes, across waves,
# that divide into no vectors, of a row that no team holds
GROUPS = [(1, 1, 1), (3, 7, 7), (2, 63, 21), (5, 40, 8), (17, 128, 128), (4, 512, 128), (4, 512, 32), (3, 264, 264), (3, 264, 24), (2, 520, 520),
          (7, 1032, 8), (2, 2056, 257), (2, 5120, 5120), (2, 5120, 128), (2, 2560, 512), (2, 5120, 1024), (1, 8200, 40), (2, 2047, 89), (2, 12296, 12296),
          (2, 12320, 32), (1, 15000, 3000), (2100, 16, 16), (600, 24, 3), (33, 96, 48)]


@pytest.mark.parametrize("rows,D,group", GROUPS)
@pytest.mark.parametrize("dtype,res", [(BF, F32), (BF, BF), (F32, F32)])
@pytest.mark.parametrize("scaled", [False, True])
def test_q8(rows, D, group, dtype, res, scaled):
    x, residual = draw((rows, D), dtype, 1), draw((rows, D), res, 2, 2.0)
    w = draw((D,), F32, 4, 0.2, 1.0)
    scale = draw((D,), F32, 6, 0.1, 0.5) if scaled else None
    q, qs, total = bd.norm_add_q8_fwd(x, residual, w, EPS, group=group, scale=scale)
    assert q.dtype == torch.float8_e4m3fn and qs.shape == (rows, D // group) and total.dtype == res
    assert rel(total, norms.norm_add_f64(x, residual, w, EPS, scale)[1]) <= torch.finfo(res).eps / 2 + 4 * U
    # from the sum as it is stored
    y = norms.norm_add_f64(total.double() * 0, total, w, EPS)[0]
    eq, es = norms.q8_of(y, group)
    t = (16 + 2 * D ** 0.5) * U
    assert bool(((qs.double() - es).abs() <= t * es).all())
    err, mag = (q.double() - eq).abs(), eq.abs()
    assert bool((err <= torch.clamp_min(mag * 2.0 ** -4, 2.0 ** -10) + 3 * t * mag).all())
    # the largest of a group is 448 to a rounding, which e4m3 holds
    assert bool((q.double().view(rows, -1, group).abs().amax(-1) == 448).all())
    # its plain sibling's sum and norm
    yp, tp = bd.norm_add_fwd(x, residual, w, EPS, scale=scale)
    assert torch.equal(total, tp)
    assert rel(q.double().view(rows, -1, group) * qs.double()[..., None], yp.double().view(rows, -1, group)) <= 2.0 ** -4 + torch.finfo(dtype).eps


def test_q8_is_the_nearest_value():
    """Away from a border by more than the sums' error, q is the nearest e4m3 value."""
    x, residual, w = draw((64, 512), F32, 1), draw((64, 512), F32, 2), draw((512,), F32, 4, 0.2, 1.0)
    q, _, total = bd.norm_add_q8_fwd(x, residual, w, EPS, group=64)
    eq, _ = norms.q8_of(norms.norm_add_f64(total * 0, total, w, EPS)[0], 64)
    values = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    values = values[values.isfinite()].unique().cuda()
    borders = (values[1:] + values[:-1]) / 2
    near = torch.searchsorted(borders, eq.contiguous())
    gap = torch.minimum((eq - borders[(near - 1).clamp_min(0)]).abs(), (eq - borders[near.clamp_max(len(borders) - 1)]).abs())
    clear = gap > 3 * (16 + 2 * 512 ** 0.5) * U * eq.abs()
    assert float(clear.double().mean()) > 0.99 and torch.equal(q.double()[clear], values[near][clear])


def test_q8_zeros_nan_and_infinity():
    x, residual, w = torch.zeros((4, 256), device="cuda"), draw((4, 256), F32, 2), torch.ones(256, device="cuda")
    residual[0] = 0.0                     # a row of zeros
    residual[1, 64:128] = 0.0             # a group of zeros
    residual[2, 3] = float("nan")
    residual[3, 200] = float("inf")
    q, qs, _ = bd.norm_add_q8_fwd(x, residual, w, EPS, group=64)
    q = q.float()
    assert bool((q[0] == 0).all()) and bool((qs[0] == 2.0 ** -126).all())
    assert bool((q[1, 64:128] == 0).all()) and float(qs[1, 1]) == 2.0 ** -126 and float(qs[1, 0]) > 1e-4
    assert bool(q[2].isnan().all()) and bool(qs[2].isnan().all())
    assert bool(qs[3, 3].isnan()) and bool(q[3, 192:].isnan().all()) and bool((q[3, :192] == 0).all())


def test_q8_in_place_other_stream_and_rows_behind():
    x, residual, w = draw((9, 640), BF, 1), draw((9, 640), F32, 2), draw((640,), F32, 3, 0.2, 1.0)
    q0, qs0, s0 = bd.norm_add_q8_fwd(x, residual, w, EPS, group=128)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    q1, qs1, s1 = bd.norm_add_q8_fwd(x, residual, w, EPS, group=128, stream=side)
    side.synchronize()
    assert torch.equal(q1.view(torch.uint8), q0.view(torch.uint8)) and torch.equal(qs1, qs0) and torch.equal(s1, s0)
    q = torch.full((12, 640), 7, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    qs = torch.full((12, 5), 7.0, device="cuda")
    bd.ssd_norm_add_q8_fwd(x, residual, None, w, residual, q[:9], qs[:9], 128, EPS)
    assert torch.equal(residual, s0) and torch.equal(q[:9].view(torch.uint8), q0.view(torch.uint8)) and torch.equal(qs[:9], qs0)
    assert bool((q[9:].view(torch.uint8) == 7).all()) and bool((qs[9:] == 7).all())
