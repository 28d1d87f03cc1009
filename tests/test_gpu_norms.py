"""The norms around a block against their float64 form (MI355X only).

Tolerances: every output is rounded once (half a step, eps / 2 of its type, relative to
the value) on top of sums in 32 bits.  A sum of n terms in 32 bits is off by at most about
sqrt(n) 2^-24 of its terms' 2-norm in the mean; a segment's two sums and the dozen
roundings of an element's chain are covered by (16 + 2 sqrt(n)) 2^-24 of the output's
2-norm.  Parameter gradients add the rows: (16 + 2 sqrt(n) + 2 sqrt(rows)) 2^-24.  The
comparison is of 2-norms over the whole output.
"""
import pytest
import torch

from oracle import norms
from selective_state_space_ssd_amd import binding as bd

pytestmark = pytest.mark.gpu
EPS = 1e-5
U = 2.0 ** -24


def rel(got, want):
    got, want = got.double(), want.double()
    assert got.shape == want.shape
    n = float(want.norm())
    d = float((got - want).norm())
    return d / n if n else d


def out_tol(dtype, n):
    return torch.finfo(dtype).eps / 2 + (16 + 2 * n ** 0.5) * U


def par_tol(n, rows):
    return (16 + 2 * n ** 0.5 + 2 * rows ** 0.5) * U


def draw(shape, dtype, seed, scale=1.0, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale + shift).to(dtype).cuda()


BF, F32 = torch.bfloat16, torch.float32

# rows, D, group: one element; odd lengths (no vectors); teams of 16, 64 and 256 lanes at
# their last length and one beyond; groups; segments that no team holds
SHAPES = [(1, 1, 1), (3, 7, 7), (5, 40, 8), (2, 63, 21), (17, 128, 128), (4, 512, 128), (3, 264, 264),
          (2, 520, 520), (7, 1032, 1032), (2, 2056, 2056), (3, 4104, 4104), (2, 5120, 5120), (1, 8200, 8200),
          (2, 2047, 2047), (2, 2051, 2051), (2, 12296, 12296), (1, 30000, 15000), (2100, 16, 16), (600, 24, 3)]


@pytest.mark.parametrize("rows,D,group", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("gate_first", [False, True])
def test_norm_gate_and_gradients(rows, D, group, dtype, gate_first):
    x, z, dy = (draw((rows, D), dtype, s) for s in (1, 2, 3))
    w = draw((D,), F32, 4, 0.2, 1.0)
    y = bd.norm_gate_fwd(x, z, w, group, EPS, gate_first)
    assert y.dtype == dtype
    assert rel(y, norms.norm_gate_f64(x, z, w, group, EPS, gate_first)) <= out_tol(dtype, group)
    dx, dz, dw = bd.norm_gate_bwd(x, z, w, dy, group, EPS, gate_first)
    ex, ez, ew = norms.norm_gate_grads_f64(x, z, w, dy, group, EPS, gate_first)
    # dx takes the part along n out: what is left may be much smaller than its terms, as
    # for a group of few elements, so its error is taken against the terms' size
    inv = 1 / torch.sqrt(((x.double() * (torch.nn.functional.silu(z.double()) if gate_first else 1)).view(rows, -1, group) ** 2).mean(-1) + EPS)
    gate = torch.nn.functional.silu(z.double())
    terms = ((dy.double() * w.double() * gate).view(rows, -1, group) * inv[..., None]).norm()
    assert float((dx.double() - ex).norm()) <= torch.finfo(dtype).eps / 2 * float(ex.norm()) + out_tol(F32, group) * float(terms) * 4
    if gate_first:     # dz is du x act': the same difference
        slope = torch.autograd.functional.jvp(torch.nn.functional.silu, z.double(), torch.ones_like(z.double()))[1]
        terms = ((dy.double() * w.double()).view(rows, -1, group) * inv[..., None] * (x.double() * slope).view(rows, -1, group)).norm()
        assert float((dz.double() - ez).norm()) <= torch.finfo(dtype).eps / 2 * float(ez.norm()) + out_tol(F32, group) * float(terms) * 4
    else:
        assert rel(dz, ez) <= out_tol(dtype, group)
    assert rel(dw, ew) <= par_tol(group, rows)


def test_norm_without_gate():
    x, dy, w = draw((6, 96), BF, 1), draw((6, 96), BF, 2), draw((96,), F32, 3, 0.2, 1.0)
    y = bd.norm_gate_fwd(x, None, w, 96, EPS)
    assert rel(y, norms.norm_gate_f64(x, None, w, 96, EPS, False)) <= out_tol(BF, 96)
    dx, dz, dw = bd.norm_gate_bwd(x, None, w, dy, 96, EPS)
    ex, _, ew = norms.norm_gate_grads_f64(x, None, w, dy, 96, EPS, False)
    assert dz is None and rel(dx, ex) <= 2 * out_tol(BF, 96) and rel(dw, ew) <= par_tol(96, 6)


@pytest.mark.parametrize("rows,D,group", SHAPES)
@pytest.mark.parametrize("dtype,res", [(BF, F32), (BF, BF), (F32, F32)])
@pytest.mark.parametrize("scaled", [False, True])
def test_norm_add_and_gradients(rows, D, group, dtype, res, scaled):
    x, dy = draw((rows, D), dtype, 1), draw((rows, D), dtype, 3)
    residual, d_sum = draw((rows, D), res, 2, 2.0), draw((rows, D), res, 5)
    w = draw((D,), F32, 4, 0.2, 1.0)
    scale = draw((D,), F32, 6, 0.1, 0.5) if scaled else None
    y, total = bd.norm_add_fwd(x, residual, w, EPS, scale=scale)
    ey, etotal = norms.norm_add_f64(x, residual, w, EPS, scale)
    assert total.dtype == res and y.dtype == dtype
    assert rel(total, etotal) <= torch.finfo(res).eps / 2 + 4 * U
    # a bf16 sum that falls next to a rounding border may be held one step off
    assert rel(y, ey) <= out_tol(dtype, D) + (4 * U if res == F32 else torch.finfo(res).eps)
    # the stored sum goes into the backward pass, on both sides
    dx, dres, dw, dscale = bd.norm_add_bwd(x, total, w, dy, d_sum, EPS, scale=scale)
    ex, eres, ew, escale = norms.norm_add_grads_f64(x, total, w, dy, d_sum, EPS, scale)
    assert rel(dx, ex) <= 2 * out_tol(dtype, D) and rel(dres, eres) <= 2 * out_tol(res, D)
    assert rel(dw, ew) <= par_tol(D, rows)
    if scaled:
        assert rel(dscale, escale) <= 2 * par_tol(D, rows)
    else:
        assert dscale is None


def test_norm_add_in_place_without_further_gradient_or_x():
    x, residual, w = draw((9, 320), BF, 1), draw((9, 320), F32, 2), draw((320,), F32, 3, 0.2, 1.0)
    y0, s0 = bd.norm_add_fwd(x, residual, w, EPS)
    y = torch.empty_like(x)
    bd.ssd_norm_add_fwd(x, residual, None, w, residual, y, EPS)
    assert torch.equal(y, y0) and torch.equal(residual, s0)
    dy = draw((9, 320), BF, 4)
    dx, dres, dw, ds = bd.norm_add_bwd(None, s0, w, dy, None, EPS)
    ex, eres, ew, _ = norms.norm_add_grads_f64(x, s0, w, dy, None, EPS)
    assert ds is None and rel(dx, ex) <= 2 * out_tol(BF, 320) and rel(dres, eres) <= 2 * out_tol(F32, 320)
    assert rel(dw, ew) <= par_tol(320, 9)


def test_rows_are_independent_of_nan_and_inf_in_others():
    x, z, w = draw((33, 128), BF, 1), draw((33, 128), BF, 2), draw((128,), F32, 3)
    y0 = bd.norm_gate_fwd(x, z, w, 128, EPS)
    x[5, 7], x[20, 0] = float("nan"), float("inf")
    y = bd.norm_gate_fwd(x, z, w, 128, EPS)
    rest = [r for r in range(33) if r not in (5, 20)]
    assert torch.equal(y[rest], y0[rest]) and y[5].isnan().all() and y[20, 0].isnan()


def test_no_rows():
    x, w = torch.empty((0, 64), dtype=BF, device="cuda"), torch.ones(64, device="cuda")
    assert bd.norm_gate_fwd(x, x, w, 64, EPS).shape == (0, 64)
    dx, dz, dw = bd.norm_gate_bwd(x, x, w, x, 64, EPS)
    assert dx.shape == (0, 64) and float(dw.abs().max()) == 0.0
    _, _, dw, ds = bd.norm_add_bwd(x, x, w, x, x, EPS, scale=w)
    assert float(dw.abs().max()) == 0.0 and float(ds.abs().max()) == 0.0


def test_parameter_gradients_repeat_and_rows_behind_stay():
    x, z, dy, w = draw((3000, 256), BF, 1), draw((3000, 256), BF, 2), draw((3000, 256), BF, 3), draw((256,), F32, 4)
    a = bd.norm_gate_bwd(x, z, w, dy, 128, EPS)
    b = bd.norm_gate_bwd(x, z, w, dy, 128, EPS)
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    big = torch.full((3010, 256), 7.0, dtype=BF, device="cuda")
    bd.ssd_norm_gate_fwd(x, z, w, big[:3000], 128, EPS, False)
    assert (big[3000:] == 7.0).all()


def test_captured_and_replayed():
    x, z, w, dy = draw((70, 512), BF, 1), draw((70, 512), BF, 2), draw((512,), F32, 3, 0.2, 1.0), draw((70, 512), BF, 4)
    outs = [torch.empty_like(x) for _ in range(3)] + [torch.empty_like(w)]
    ws = torch.empty(bd.ssd_norm_bwd_workspace_bytes(70, 512, 512, 1, bd.SSD_DTYPE_BF16), dtype=torch.uint8, device="cuda")

    def step():
        bd.ssd_norm_gate_fwd(x, z, w, outs[0], 512, EPS, True)
        bd.ssd_norm_gate_bwd(x, z, w, dy, outs[1], outs[2], outs[3], 512, EPS, True, ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        x.copy_(draw((70, 512), BF, 10 + seed))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(s, t) for s, t in zip(got, outs))


def test_on_another_stream():
    x, z, w = draw((64, 640), BF, 1), draw((64, 640), BF, 2), draw((640,), F32, 3)
    want = bd.norm_gate_fwd(x, z, w, 640, EPS)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = bd.norm_gate_fwd(x, z, w, 640, EPS, stream=side)
    side.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_parameter_gradients_without_eps(dtype):
    """eps = 0 and more rows than the backward pass has blocks, not a multiple of them: the
    blocks without a row in the last turn add nothing."""
    rows, D = 1500, 520
    x, z, dy = (draw((rows, D), dtype, s) for s in (1, 2, 3))
    w = draw((D,), F32, 4, 0.2, 1.0)
    for gate_first in (False, True):
        _, _, dw = bd.norm_gate_bwd(x, z, w, dy, D, 0.0, gate_first)
        assert rel(dw, norms.norm_gate_grads_f64(x, z, w, dy, D, 0.0, gate_first)[2]) <= par_tol(D, rows)
    scale = draw((D,), F32, 6, 0.1, 0.5)
    _, _, dw, dscale = bd.norm_add_bwd(x, x, w, dy, None, 0.0, scale=scale)
    _, _, ew, escale = norms.norm_add_grads_f64(x, x, w, dy, None, 0.0, scale)
    assert rel(dw, ew) <= par_tol(D, rows) and rel(dscale, escale) <= 2 * par_tol(D, rows)
