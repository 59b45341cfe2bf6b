"""The norm with the residual's addition, its int8 output and its gradients
against the formulas in 64 bits: types, one row to many, lengths a lane holds and
does not, rows in place, rows of zeros and rows that are not finite.

Tolerances, in units of 2^-24: h one rounding; its mean square (each lane adds
cols / 256 squares at least, cols / 64 at most, and 8 steps more) below cols / 64 + 16
units, halved by the root; y four more roundings; then half a step of bf16."""
import pytest
import torch

import quantize_precision_gemm_amd as q

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = 1e-6
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def randn(seed, *shape):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV)


def pitched(t, more):
    wide = torch.full((t.shape[0], t.shape[1] + more), 3.0, dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def inputs(rows, cols, x, s, w, residual, more=0):
    scale = torch.exp(0.5 * randn(9, 1, cols)) * torch.exp(randn(8, rows, 1))
    return (pitched((randn(1, rows, cols) * scale).to(x), more), pitched((2 * randn(2, rows, cols)).to(s), more) if residual else None,
            (1 + 0.2 * randn(3, cols)).to(w) if w else None)


def units(cols):
    return (cols / 64 + 16) / 2 + 6


CASES = [(1, 16), (3, 64), (5, 80), (1000, 128), (37, 112), (9, 144), (301, 256), (17, 272), (600, 512), (9, 528), (2, 1024), (700, 2048), (4, 2048), (33, 2064), (1, 5120), (65, 5120), (3, 8192),
         (5, 8208), (2, 16384), (2, 20000)]
TYPES = [(BF, BF, BF, True), (F32, BF, F32, True), (BF, F32, F32, True), (F32, F32, BF, True), (BF, BF, F32, False), (F32, BF, None, False)]


@pytest.mark.parametrize("rows,cols", CASES)
@pytest.mark.parametrize("x,s,w,residual", TYPES)
def test_norm(rows, cols, x, s, w, residual):
    xs, r, weight = inputs(rows, cols, x, s, w, residual, 16 if rows % 2 else 0)
    y, h = q.nvfp4_rmsnorm(xs, weight, EPS, residual=r)
    want_h = xs.double() + (r.double() if residual else 0.0)
    if residual:
        assert h.dtype == s and ((h.double() - want_h).abs() <= (HALF[s] * 1.001 + U) * want_h.abs()).all()
    else:
        assert h is None
    want = want_h / torch.sqrt(want_h.square().mean(1, keepdim=True) + EPS)
    if weight is not None:
        want = want * weight.double()
    # (where x and the residual cancel, h's rounding is still a unit of h)
    assert ((y.double() - want).abs() <= (2.0 ** -8 * 1.001 + units(cols) * U) * want.abs()).all()
    if residual and x == s:  # the sum where the residual lay, and where x lay
        for place in (0, 1):
            a, b = xs.clone(), r.clone()
            y2, h2 = q.nvfp4_rmsnorm(a, weight, EPS, residual=b, h=(a, b)[place])
            assert h2 is (a, b)[place] and torch.equal(h2, h) and torch.equal(y2, y)
            assert torch.equal((b, a)[place], (r, xs)[place])


@pytest.mark.parametrize("rows,cols", CASES)
@pytest.mark.parametrize("x,s,w,residual", TYPES)
def test_norm_int8(rows, cols, x, s, w, residual):
    xs, r, weight = inputs(rows, cols, x, s, w, residual, 16 if rows % 2 else 0)
    place = r.clone() if residual else None
    y, h = q.nvfp4_rmsnorm_i8(xs, weight, EPS, residual=place, h=place)
    if residual:
        assert torch.equal(h, q.nvfp4_rmsnorm(xs, weight, EPS, residual=r)[1])
    want = xs.double() + (r.double() if residual else 0.0)
    want = want / torch.sqrt(want.square().mean(1, keepdim=True) + EPS) * (weight.double() if weight is not None else 1.0)
    top = want.abs().amax(1)
    assert ((y.scales.double() - top / 127).abs() <= (units(cols) + 2) * U * top / 127).all()
    exact = want * 127 / top[:, None]
    # a code is the nearest whole number, or the other one where the quotient lies as near to a half as it is off
    off = (y.codes.double() - exact).abs()
    assert (off <= 0.5 + 127 * (2 * units(cols) + 8) * U).all()
    assert (y.codes.abs().amax(1) == 127).all()


def test_the_int8_rows_feed_the_int8_product():
    x, r, weight = inputs(37, 1296, BF, BF, BF, True)
    w8 = q.nvfp4_i8_quantize((0.02 * randn(5, 504, 1296)).bfloat16())
    y8, _ = q.nvfp4_rmsnorm_i8(x, weight, EPS, residual=r)
    got = q.nvfp4_i8_gemm(y8, w8, F32)
    acc = y8.codes.double() @ w8.codes.double().t()
    want = acc * y8.scales.double()[:, None] * w8.scales.double()[None]
    assert ((got.double() - want).abs() <= 3 * U * want.abs()).all()


@pytest.mark.parametrize("cols", [64, 5120, 8208])
def test_rows_of_zeros_tiny_and_not_finite(cols):
    x = randn(1, 8, cols)
    x[0] = 0.0
    x[1] = 1e-38 * x[1]
    x[2, 7] = torch.nan
    x[3, 9] = torch.inf
    x[4] = 1e-12 * x[4]
    y, _ = q.nvfp4_rmsnorm(x, None, EPS)
    assert (y[0] == 0).all() and torch.isnan(y[2]).all() and torch.isnan(y[3, 9]) and (y[3, :9] == 0).all()
    assert torch.isfinite(y[5:]).all() and torch.isfinite(y[1]).all()
    y8, _ = q.nvfp4_rmsnorm_i8(x, None, EPS)
    assert (y8.codes[0] == 0).all() and y8.scales[0] == 0
    for row in (2, 3):
        assert not torch.isfinite(y8.scales[row]) and (y8.codes[row] == 0).all()
    # scales next to the smallest numbers: codes as of any other row
    for row in (1, 4):
        want = x[row].double()
        top = want.abs().max()
        assert (y8.codes[row].double() - want * 127 / top).abs().max() <= 0.51
    # no eps: a row of tiny numbers is normalised like any other, one of zeros is not a number
    tiny = (x[5:6] * 1e-15).contiguous()
    got = q.nvfp4_rmsnorm(tiny, None, 0.0)[0].double()
    want = tiny.double() / tiny.double().square().mean().sqrt()
    assert ((got - want).abs() <= 2.0 ** -7 * want.abs()).all()
    assert torch.isnan(q.nvfp4_rmsnorm(x[:1], None, 0.0)[0]).all()
    assert (q.nvfp4_rmsnorm(x[:1], None, 1e-300)[0] == 0).all()  # (an eps below fp32's range is not 0)


BACK = [(1, 16), (3, 64), (5, 72), (1000, 128), (130, 120), (9, 136), (301, 256), (2100, 192), (17, 264), (600, 512), (9, 520), (700, 1024), (4, 1032), (300, 2048), (1, 5120), (65, 5120), (700, 2568), (3, 8200),
        (520, 128), (2, 16384), (5000, 256)]


@pytest.mark.parametrize("rows,cols", BACK)
@pytest.mark.parametrize("d,s,w,dh,out", [(BF, BF, F32, True, BF), (F32, F32, BF, True, F32), (BF, F32, F32, False, BF),
                                          (F32, BF, None, True, F32), (BF, BF, BF, False, F32)])
def test_backward(rows, cols, d, s, w, dh, out):
    h, _, weight = inputs(rows, cols, s, s, w, False, 8 if rows % 2 else 0)
    dy = pitched(randn(4, rows, cols).to(d), 8 if rows % 2 else 0)
    along = randn(5, rows, cols).to(s) if dh else None
    dx, dw = q.nvfp4_rmsnorm_backward(dy, h, weight, EPS, dh=along, out_dtype=out)
    x = h.double().requires_grad_()
    wd = (weight.double() if w else torch.ones(cols, dtype=torch.float64, device=DEV)).requires_grad_()
    y = x / torch.sqrt(x.square().mean(1, keepdim=True) + EPS) * wd
    want, want_w = torch.autograd.grad(y, (x, wd), dy.double())
    rstd = 1 / torch.sqrt(h.double().square().mean(1, keepdim=True) + EPS)
    u, xhat = dy.double() * wd.detach(), h.double() * rstd
    # sizes of the terms: rstd |u|, rstd |xhat| mean|u xhat|
    size = rstd * (u.abs() + xhat.abs() * (u * xhat).abs().mean(1, keepdim=True))
    if dh:
        want, size = want + along.double(), size + along.double().abs()
    assert dx.dtype == out
    assert ((dx.double() - want).abs() <= HALF[out] * 1.001 * want.abs() + (3 * units(cols) + 8) * U * size).all()
    if w is None:
        assert dw is None
    else:
        # a column's sum: rows over the groups, then groups in runs; each term's own rounding on top
        steps = rows / 256 + 128 + 2 * units(cols)
        assert ((dw.double() - want_w).abs() <= steps * U * (dy.double() * xhat).abs().sum(0) + 1e-30).all()
    # a difference quotient of the formula along one direction
    e = randn(6, rows, cols).double()

    def value(t):
        z = h.double() + t * e
        return (z / torch.sqrt(z.square().mean(1, keepdim=True) + EPS) * wd.detach() * dy.double()).sum()
    step = 1e-5 * h.double().abs().mean()
    slope = (value(step) - value(-step)) / (2 * step) + ((along.double() * e).sum() if dh else 0.0)
    bound = ((HALF[out] * 1.01 * want.abs() + (3 * units(cols) + 8) * U * size + 1e-6 * size) * e.abs()).sum()
    assert abs((dx.double() * e).sum() - slope) <= bound


def test_backward_in_place_and_again():
    """dx where dy or dh lay; the same bits in every call, with a workspace of one's own."""
    rows, cols = 333, 2568
    h, _, weight = inputs(rows, cols, BF, BF, F32, False)
    dy, dh = randn(4, rows, cols).bfloat16(), randn(5, rows, cols).bfloat16()
    ws = torch.empty(q.nvfp4_rmsnorm_backward_workspace(rows, cols), dtype=torch.uint8, device=DEV)
    dx, dw = q.nvfp4_rmsnorm_backward(dy, h, weight, EPS, dh=dh, workspace=ws)
    for place in (0, 1):
        a, b = dy.clone(), dh.clone()
        got, w = q.nvfp4_rmsnorm_backward(a, h, weight, EPS, dh=b, out=(a, b)[place], workspace=ws)
        assert torch.equal(got, dx) and torch.equal(w, dw)
    with pytest.raises(ValueError):
        q.nvfp4_rmsnorm_backward(dy, h, weight, EPS, workspace=ws[:-16])


def test_empty_and_refusals():
    none = torch.empty(0, 64, dtype=BF, device=DEV)
    w = torch.ones(64, device=DEV)
    assert q.nvfp4_rmsnorm(none, w)[0].shape == (0, 64) and q.nvfp4_rmsnorm_i8(none, w)[0].codes.shape == (0, 64)
    dx, dw = q.nvfp4_rmsnorm_backward(none, none, w)
    assert dx.shape == (0, 64) and (dw == 0).all() and dw.shape == (64,)
    thin = torch.empty(3, 0, dtype=BF, device=DEV)
    answer = q.nvfp4_rmsnorm_i8(thin)[0]
    assert q.nvfp4_rmsnorm(thin)[0].shape == (3, 0) and answer.codes.shape == (3, 0) and (answer.scales == 0).all()
    x = randn(1, 4, 64).bfloat16()
    with pytest.raises(TypeError):
        q.nvfp4_rmsnorm(x.half())
    with pytest.raises(ValueError):
        q.nvfp4_rmsnorm(x, w[:32])
    with pytest.raises(ValueError):
        q.nvfp4_rmsnorm(x, w, residual=x[:3])
    with pytest.raises(TypeError):
        q.nvfp4_rmsnorm(x, w, residual=x, h=torch.empty(4, 64, device=DEV))
    with pytest.raises(TypeError):
        q.nvfp4_rmsnorm(x, w, out=torch.empty(4, 64, device=DEV))
    with pytest.raises(RuntimeError):
        q.nvfp4_rmsnorm(x[:, :60].contiguous(), None)
    with pytest.raises(RuntimeError):
        q.nvfp4_rmsnorm(x, w, eps=-1.0)
    with pytest.raises(RuntimeError):
        q.nvfp4_rmsnorm_i8(x[:, :56].contiguous())
    with pytest.raises(TypeError):
        q.nvfp4_rmsnorm_backward(x, x, w, dh=x.float())
    with pytest.raises(ValueError):
        q.nvfp4_rmsnorm_backward(x, x[:2], w)
