"""The residual norm with dropout over many rows, with the row lengths of each of its backward
teams, and past 2^31 elements (MI355X only).  Tolerances as in test_gpu_norm_drop_q8."""
import pytest
import torch

from oracle import norms
from selective_state_space_ssd_amd import binding as bd
from test_gpu_norms import BF, EPS, F32, U, draw, out_tol, par_tol, rel

pytestmark = pytest.mark.gpu


def state(seed, offset):
    return torch.tensor([seed, offset], dtype=torch.int64, device="cuda")


# more rows than blocks, not a multiple of them: teams of 16 and 64 lanes, of a block's four
# waves, of five to eight waves (bf16) and the first length beyond
@pytest.mark.parametrize("rows,D", [(9001, 128), (4100, 512), (1500, 1024), (1300, 2056), (1100, 2560), (700, 4096), (600, 4104)])
@pytest.mark.parametrize("dtype,res", [(BF, F32), (F32, F32)])
@pytest.mark.parametrize("eps", [0.0, EPS])
def test_gradients_over_many_rows(rows, D, dtype, res, eps):
    x, dy = draw((rows, D), dtype, 1), draw((rows, D), dtype, 3)
    residual, d_sum = draw((rows, D), res, 2, 2.0), draw((rows, D), res, 5)
    w, scale = draw((D,), F32, 4, 0.2, 1.0), draw((D,), F32, 6, 0.1, 0.5)
    rng = (7, 1 << 33)
    factor = norms.dropout_factor((rows, D), 0.2, rng).cuda()
    _, total = bd.norm_add_drop_fwd(x, residual, w, eps, 0.2, state(*rng), scale=scale)
    first = bd.norm_add_drop_bwd(x, total, w, dy, d_sum, eps, 0.2, state(*rng), scale=scale)
    dx, dres, dw, dscale = first
    ex, eres, ew, escale = norms.norm_add_grads_f64(x.double() * factor, total, w, dy, d_sum, eps, scale)
    assert rel(dx, ex * factor) <= 2 * out_tol(dtype, D) and rel(dres, eres) <= 2 * out_tol(res, D)
    assert rel(dw, ew) <= par_tol(D, rows) and rel(dscale, escale) <= 2 * par_tol(D, rows)
    again = bd.norm_add_drop_bwd(x, total, w, dy, d_sum, eps, 0.2, state(*rng), scale=scale)
    assert all(torch.equal(s, t) for s, t in zip(first, again))


def test_offsets_past_31_bits():
    """2^20 + 3 rows of 2056 channels: the last rows' mask, sum, norm and gradients."""
    rows, D, n = (1 << 20) + 3, 2056, 5
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty((rows, D), dtype=BF, device="cuda").normal_(generator=g)
    w = torch.rand(D, generator=g, device="cuda") + 0.5
    residual = torch.zeros((rows, D), dtype=BF, device="cuda")
    y, total = bd.norm_add_drop_fwd(x, residual, w, EPS, 0.25, state(3, 4))
    # the words of the last rows' elements: the whole mask would take as long as all else
    at = (rows - n) * D
    assert at % 4 == 0 and at > 1 << 31
    words = norms.philox_words(n * D, 3, 4, first=at)
    factor = (torch.from_numpy(words.astype("int64")) >= 1 << 30).view(n, D).cuda() / 0.75
    ey, etotal = norms.norm_add_f64(x[-n:].double() * factor, residual[-n:], w, EPS)
    assert torch.equal(total[-n:] != 0, (factor != 0) & (x[-n:] != 0))
    assert rel(total[-n:], etotal) <= torch.finfo(BF).eps / 2 + 6 * U and rel(y[-n:], ey) <= out_tol(BF, D) + torch.finfo(BF).eps
    del residual
    dx, dres, dw, _ = bd.norm_add_drop_bwd(None, total, w, y, None, EPS, 0.25, state(3, 4))
    ex, eres, _, _ = norms.norm_add_grads_f64(x[-n:], total[-n:], w, y[-n:], None, EPS)
    assert rel(dres[-n:], eres) <= 2 * out_tol(BF, D) and bool((dx[-n:][factor == 0] == 0).all())
    assert rel(dx[-n:], ex * factor) <= 2 * out_tol(BF, D)
    del dx, dres, y
    q, qs, s = bd.norm_add_q8_fwd(x, total, w, EPS, group=257)
    eq, es = norms.q8_of(norms.norm_add_f64(s[-n:].double() * 0, s[-n:], w, EPS)[0], 257)
    t = (16 + 2 * D ** 0.5) * U
    assert bool(((qs[-n:].double() - es).abs() <= t * es).all())
    assert bool(((q[-n:].double() - eq).abs() <= torch.clamp_min(eq.abs() * 2.0 ** -4, 2.0 ** -10) + 3 * t * eq.abs()).all())


@pytest.mark.parametrize("rows,D,group", [(5, 40, 1), (3, 2056, 1), (4, 520, 2), (4, 520, 4), (2, 4104, 3), (2, 4104, 1), (1, 12296, 2), (70, 128, 16), (9, 4096, 256), (9, 4096, 2048),
                                          (1030, 2560, 128)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_q8_groups_of_few_and_many_channels(rows, D, group, dtype):
    x, residual, w = draw((rows, D), dtype, 1), draw((rows, D), F32, 2, 2.0), draw((D,), F32, 4, 0.2, 1.0)
    q, qs, total = bd.norm_add_q8_fwd(x, residual, w, EPS, group=group)
    eq, es = norms.q8_of(norms.norm_add_f64(total.double() * 0, total, w, EPS)[0], group)
    t = (16 + 2 * D ** 0.5) * U
    assert bool(((qs.double() - es).abs() <= t * es).all())
    assert bool(((q.double() - eq).abs() <= torch.clamp_min(eq.abs() * 2.0 ** -4, 2.0 ** -10) + 3 * t * eq.abs()).all())
    assert bool((q.double().view(rows, -1, group).abs().amax(-1) == 448).all())
