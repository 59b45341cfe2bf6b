"""A product with bias, activation and residual in its epilogue, dense and
grouped by expert, and the gradients through it, against the formulas in 64 bits:
each kernel (few rows, 128 and 256 tiles, split contractions), odd sizes,
experts without rows, rows of no expert, types, pitches, in place.

Tolerances: a sum of K products in fp32 rounds by at most (K / 16 + 40) 2^-24 of
the sum of their sizes (16 or 32 products an instruction, partial sums in order),
an activation changes it by its slope (at most 2 |z| for relu2, 1.13 for gelu) and 8 units more,
then half a step of the output's type."""
import pytest
import torch

import quantize_precision_gemm_amd as q

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}
ACTS = {q.ACT_NONE: lambda z: z, q.ACT_RELU2: lambda z: torch.relu(z) ** 2, q.ACT_SILU: torch.nn.functional.silu,
        q.ACT_GELU: lambda z: torch.nn.functional.gelu(z, approximate="tanh")}


def randn(seed, *shape):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV)


def pitched(t, more):
    wide = torch.full((t.shape[0], t.shape[1] + more), 3.0, dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def slope_bound(act, z, dz):
    if act == q.ACT_RELU2:
        return 2 * z.abs() * dz + dz * dz
    return 1.2 * dz


def reference(x, w, ends, bias):
    """(z, the sum of the sizes of what it adds up), rows of no expert zero."""
    T, N = x.shape[0], w.shape[-2]
    z, size = torch.zeros(T, N, dtype=torch.float64, device=DEV), torch.zeros(T, N, dtype=torch.float64, device=DEV)
    begin = 0
    for e, end in enumerate([T] if ends is None else ends):
        we = (w if ends is None else w[e]).double()
        rows = x[begin:end].double()
        z[begin:end], size[begin:end] = rows @ we.t(), rows.abs() @ we.t().abs()
        if bias is not None:
            b = (bias if ends is None else bias[e]).double()
            z[begin:end] += b
            size[begin:end] += b.abs()
        begin = end
    return z, size, begin


def check(T, N, K, ends, act, bias_dtype, residual, pre, out, more=0, seed=0, **how):
    x = pitched(randn(seed + 1, T, K).bfloat16(), 2 * more)
    lead = () if ends is None else (len(ends),)
    w = (randn(seed + 2, *lead, N, K) * max(K, 1) ** -0.5).bfloat16()
    bias = randn(seed + 3, *lead, N).to(bias_dtype) if bias_dtype else None
    r = pitched(randn(seed + 4, T, N).to(out), more) if residual else None
    dev_ends = None if ends is None else torch.tensor(ends, dtype=torch.int32, device=DEV)
    got = q.nvfp4_bf16_linear(x, w, ends=dev_ends, bias=bias, activation=act, residual=r, with_pre=pre, out_dtype=out, **how)
    y, p = got if pre else (got, None)
    z, size, used = reference(x, w, ends, bias)
    dz = (K / 16 + 40) * U * size
    if pre:
        assert p.dtype == BF and ((p.double() - z).abs() <= dz + 2.0 ** -8 * 1.001 * z.abs()).all()
    want = ACTS[act](z)
    off = slope_bound(act, z, dz) + 8 * U * (want.abs() + z.abs())
    if residual:
        want = want + r.double()
        off = off + U * want.abs()
    want[used:] = 0.0
    off[used:] = 0.0
    assert y.dtype == out and ((y.double() - want).abs() <= off + HALF[out] * 1.001 * want.abs()).all()
    return x, w, dev_ends, bias, r, y, p


DENSE = [(1, 8, 8), (1, 2048, 1024), (3, 136, 264), (16, 512, 5120), (37, 1296, 520), (64, 1024, 2048), (100, 72, 4096), (130, 264, 1032),
         (300, 1280, 1288), (777, 1024, 512), (1000, 2056, 776), (2048, 2560, 640),
         (9, 4104, 264), (16, 5120, 1032), (20, 4120, 2048), (33, 4224, 72), (37, 6152, 1288), (64, 5128, 640),
         (16, 8200, 520), (20, 8192, 1032), (64, 10248, 264)]


@pytest.mark.parametrize("T,N,K", DENSE)
@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("out", [BF, F32])
def test_dense(T, N, K, act, out):
    check(T, N, K, None, act, F32 if T % 2 else BF, N % 16 == 0, K % 16 == 0, out, more=4 if T % 3 == 0 else 0)


@pytest.mark.parametrize("bias,residual,pre", [(b, r, p) for b in (None, BF, F32) for r in (False, True) for p in (False, True)])
@pytest.mark.parametrize("T", [5, 200, 1500])
def test_what_may_be_left_out(T, bias, residual, pre):
    check(T, 392, 520, None, q.ACT_SILU, bias, residual, pre, BF, more=8)
    check(T, 392, 520, [0, T // 3, T // 3, T], q.ACT_GELU, bias, residual, pre, F32, more=8)


GROUPED = [(16, 2048, 1024, [2, 2, 5, 9, 9, 9, 12, 16]), (40, 136, 264, [40, 40, 40]), (40, 136, 264, [0, 0, 40]), (500, 648, 520, [100, 101, 430]),
           (1000, 1288, 264, [0, 300, 300, 640, 641, 900]), (3000, 1024, 520, [1000, 1100, 2900, 3000]), (5, 64, 64, [1, 1, 1]),
           (600, 512, 64, [13, 600] + [600] * 70), (700, 256, 2048, [650]), (2048, 520, 1288, [1024, 1025, 2000])]


@pytest.mark.parametrize("T,N,K,ends", GROUPED)
@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("out", [BF, F32])
def test_grouped(T, N, K, ends, act, out):
    check(T, N, K, ends, act, BF if T % 2 else F32, True, True, out)


@pytest.mark.parametrize("K", [4096, 5120])
@pytest.mark.parametrize("ends", [None, [100, 128]])
def test_split_contraction(K, ends):
    """Few tiles and a long contraction: with a workspace the sums are taken in parts, without one whole."""
    need = q.nvfp4_bf16_grouped_gemm_workspace(q.FPROP, 1 if ends is None else 2, 128, 1024, K)
    assert need > 0
    for ws in (None, torch.empty(0, dtype=torch.uint8, device=DEV), torch.full((need,), 255, dtype=torch.uint8, device=DEV)):
        check(128, 1024, K, ends, q.ACT_GELU, F32, True, True, BF, workspace=ws)


@pytest.mark.parametrize("T,ends", [(20, None), (300, None), (1300, None), (300, [10, 200, 300])])
def test_whole_numbers(T, ends):
    """Small whole numbers: every sum is exact, so the outputs are the formula's bits."""
    g = torch.Generator(device=DEV)
    g.manual_seed(T)
    def ints(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g, device=DEV)
    N, K = 328, 456
    lead = () if ends is None else (len(ends),)
    x, w = ints(-3, 4, T, K).bfloat16(), ints(-3, 4, *lead, N, K).bfloat16()
    bias, r = ints(-9, 10, *lead, N).float(), ints(-9, 10, T, N).float()
    dev_ends = None if ends is None else torch.tensor(ends, dtype=torch.int32, device=DEV)
    z = reference(x, w, ends, bias)[0]
    y, pre = q.nvfp4_bf16_linear(x, w, ends=dev_ends, bias=bias, activation=q.ACT_RELU2, residual=r, with_pre=True, out_dtype=F32)
    assert torch.equal(y, (torch.relu(z) ** 2 + r.double()).float()) and torch.equal(pre, z.bfloat16())
    plain = q.nvfp4_bf16_linear(x, w, ends=dev_ends, out_dtype=F32)
    assert torch.equal(plain.double(), reference(x, w, ends, None)[0])


def test_no_contraction_no_experts_no_rows():
    bias = randn(1, 64)
    x0, w0 = torch.empty(10, 0, dtype=BF, device=DEV), torch.empty(64, 0, dtype=BF, device=DEV)
    assert torch.equal(q.nvfp4_bf16_linear(x0, w0, bias=bias, out_dtype=F32), bias.expand(10, 64))
    ends = torch.empty(0, dtype=torch.int32, device=DEV)
    y = q.nvfp4_bf16_linear(randn(1, 10, 64).bfloat16(), torch.empty(0, 32, 64, dtype=BF, device=DEV), ends=ends, out_dtype=F32,
                            residual=randn(2, 10, 32))
    assert (y == 0).all()
    assert q.nvfp4_bf16_linear(torch.empty(0, 64, dtype=BF, device=DEV), randn(1, 32, 64).bfloat16()).shape == (0, 32)


def test_ends_out_of_order_or_range():
    """Read as their running maximum within the rows, as the grouped products do; rows behind them get zeros."""
    T, N, K = 120, 64, 72
    x, w, bias = randn(1, T, K).bfloat16(), randn(2, 4, N, K).bfloat16(), randn(3, 4, N)
    raw = torch.tensor([-5, 60, 30, 90], dtype=torch.int32, device=DEV)
    fine = torch.tensor([0, 60, 60, 90], dtype=torch.int32, device=DEV)
    for r, f in ((raw, fine), (torch.tensor([50, 1 << 30, 3, -1], dtype=torch.int32, device=DEV),
                               torch.tensor([50, 120, 120, 120], dtype=torch.int32, device=DEV))):
        a = q.nvfp4_bf16_linear(x, w, ends=r, bias=bias, activation=q.ACT_SILU, with_pre=True)
        b = q.nvfp4_bf16_linear(x, w, ends=f, bias=bias, activation=q.ACT_SILU, with_pre=True)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        dy = randn(4, T, N).bfloat16()
        outs = [torch.full((T, N), 9.0, dtype=BF, device=DEV) for _ in range(2)]
        c = q.nvfp4_bf16_linear_backward(dy, b[1], q.ACT_SILU, ends=r, out=outs[0])
        d = q.nvfp4_bf16_linear_backward(dy, b[1], q.ACT_SILU, ends=f, out=outs[1])
        assert torch.equal(c[0], d[0]) and torch.equal(c[1], d[1])
        assert (c[0][int(f[-1]):] == 9).all()


def test_in_place():
    x, w, _, bias, r, y, pre = check(333, 264, 136, None, q.ACT_GELU, F32, True, True, BF)
    assert torch.equal(q.nvfp4_bf16_linear(x, w, bias=bias, activation=q.ACT_GELU, residual=r, out=r), y)
    dy = randn(5, 333, 264).bfloat16()
    want, db = q.nvfp4_bf16_linear_backward(dy, pre, q.ACT_GELU)
    a = dy.clone()
    assert torch.equal(q.nvfp4_bf16_linear_backward(a, pre, q.ACT_GELU, out=a)[0], want)
    b = pre.clone()
    got = q.nvfp4_bf16_linear_backward(dy, b, q.ACT_GELU, out=b)
    assert torch.equal(got[0], want) and torch.equal(got[1], db)


BACK = [(1, 8, None), (7, 520, None), (300, 1288, None), (4000, 264, None), (9000, 64, None), (16, 2048, [2, 2, 5, 9, 9, 16]),
        (500, 648, [100, 101, 430]), (3000, 1032, [0, 0, 1000, 1100, 2900, 3000]), (5, 64, [1, 1, 1]), (5000, 72, [13, 5000] + [5000] * 70),
        (5000, 16, list(range(0, 4900, 7))), (40, 136, [0, 0])]


@pytest.mark.parametrize("T,N,ends", BACK)
@pytest.mark.parametrize("act", [q.ACT_RELU2, q.ACT_SILU, q.ACT_GELU, q.ACT_NONE])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_backward(T, N, ends, act, dtype):
    """Slopes are within 16 units of their terms' sizes; a bias's sum adds a run's rows one by one, then runs in four parts."""
    more = 8 if T % 2 else 0
    pre, dy = pitched((2 * randn(1, T, N)).bfloat16(), more), pitched(randn(2, T, N).to(dtype), more)
    out = pitched(torch.full((T, N), 9.0, dtype=BF, device=DEV), more)
    dev_ends = None if ends is None else torch.tensor(ends, dtype=torch.int32, device=DEV)
    dpre, db = q.nvfp4_bf16_linear_backward(dy, pre, act, ends=dev_ends, out=out)
    z = pre.double().requires_grad_()
    slope, = torch.autograd.grad(ACTS[act](z).sum(), z)
    want, size = slope * dy.double(), (slope.abs() + 2.0) * dy.double().abs()
    used = T if ends is None else ends[-1]
    assert ((dpre.double() - want).abs()[:used] <= (2.0 ** -8 * 1.001 * want.abs() + 16 * U * size)[:used]).all()
    assert (dpre[used:] == 9).all()
    begin, steps = 0, max(8, T / 4096 + 1) + 4096 / 4 + 20
    for e, end in enumerate([T] if ends is None else ends):
        got = db if ends is None else db[e]
        assert ((got.double() - want[begin:end].sum(0)).abs() <= steps * U * size[begin:end].sum(0) + 1e-30).all()
        begin = end
    # a difference quotient of the activation along one direction
    d, h = randn(3, T, N).double(), 1e-5
    rise = (ACTS[act](pre.double() + h * d) - ACTS[act](pre.double() - h * d)) / (2 * h)
    bound = ((2.0 ** -7 * want.abs() + 16 * U * size) * d.abs())[:used].sum() + 1e-6 * (size * d.abs()).sum()
    assert abs((dpre.double() * d)[:used].sum() - (rise * dy.double())[:used].sum()) <= bound


def test_backward_without_bias_or_activation():
    dy, pre = randn(1, 50, 64).bfloat16(), randn(2, 50, 64).bfloat16()
    full = q.nvfp4_bf16_linear_backward(dy, pre, q.ACT_SILU)
    alone, none = q.nvfp4_bf16_linear_backward(dy, pre, q.ACT_SILU, with_bias=False)
    assert none is None and torch.equal(alone, full[0])
    same, db = q.nvfp4_bf16_linear_backward(dy, None)
    assert same is dy and torch.allclose(db.double(), dy.double().sum(0), rtol=0, atol=1e-4)
    assert q.nvfp4_bf16_linear_backward(dy, None, with_bias=False) == (dy, None)
    d, b = q.nvfp4_bf16_linear_backward(torch.empty(0, 64, dtype=BF, device=DEV), torch.empty(0, 64, dtype=BF, device=DEV), q.ACT_GELU)
    assert d.shape == (0, 64) and (b == 0).all()
    with pytest.raises(ValueError):
        q.nvfp4_bf16_linear_backward(dy, None, q.ACT_SILU)


@pytest.mark.parametrize("act", [q.ACT_RELU2, q.ACT_SILU, q.ACT_GELU])
def test_far_values(act):
    """Activations and slopes of large and tiny values, and of NaN."""
    v = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 1e-3, 20.0, -20.0, 88.0, -88.0, 200.0, -200.0, 3e4, -3e4, 1e19, -1e19], device=DEV)
    v = torch.cat([v, torch.full((1,), torch.nan, device=DEV)]).bfloat16()
    pre = v.repeat(3, 1)
    dz, _ = q.nvfp4_bf16_linear_backward(torch.ones(3, 16, dtype=BF, device=DEV), pre, act)
    z = v[:15].double().requires_grad_()
    want, = torch.autograd.grad(ACTS[act](z).sum(), z)
    assert ((dz[0, :15].double() - want).abs() <= 2.0 ** -8 * 1.01 * want.abs() + 2.0 ** -20).all() and torch.isnan(dz[:, 15]).all()
    bias = v.float()
    got = q.nvfp4_bf16_linear(torch.zeros(2, 8, dtype=BF, device=DEV), torch.zeros(16, 8, dtype=BF, device=DEV), bias=bias, activation=act,
                              out_dtype=F32)
    want = ACTS[act](v[:15].double())
    # 1 / (1 + e^-z) below 2^-126 (z below -87.3) may count as 0: z times that is at most |z| 2^-126 off;
    # and what itself lies below 2^-126 (1e-30 squared) may be 0
    assert ((got[0, :15].double() - want).abs() <= 2.0 ** -20 * want.abs() + 2.0 ** -126 * (1 + v[:15].double().abs())).all()
    assert torch.isnan(got[:, 15]).all()


def test_refusals():
    x, w = randn(1, 4, 64).bfloat16(), randn(2, 32, 64).bfloat16()
    ends = torch.tensor([2, 4], dtype=torch.int32, device=DEV)
    w3, x40 = torch.stack([w, w]), randn(3, 40, 64).bfloat16()
    for call, error in (
            (lambda: q.nvfp4_bf16_linear(x.float(), w), TypeError), (lambda: q.nvfp4_bf16_linear(x, w3), TypeError),
            (lambda: q.nvfp4_bf16_linear(x, w, ends=ends), TypeError), (lambda: q.nvfp4_bf16_linear(x, w3[:1], ends=ends), ValueError),
            (lambda: q.nvfp4_bf16_linear(x[:, :32], w), ValueError), (lambda: q.nvfp4_bf16_linear(x, w[:, :56]), ValueError),
            (lambda: q.nvfp4_bf16_linear(x, w[:20]), ValueError), (lambda: q.nvfp4_bf16_linear(x, w, bias=randn(1, 64)), ValueError),
            (lambda: q.nvfp4_bf16_linear(x, w, bias=randn(1, 32).half()), TypeError),
            (lambda: q.nvfp4_bf16_linear(x, w3, ends=ends, bias=randn(1, 32)), ValueError),
            (lambda: q.nvfp4_bf16_linear(x, w, residual=randn(1, 4, 32)), TypeError),
            (lambda: q.nvfp4_bf16_linear(x, w, residual=randn(1, 3, 32).bfloat16()), ValueError),
            (lambda: q.nvfp4_bf16_linear(x, w, pre=torch.empty(4, 32, device=DEV)), TypeError),
            (lambda: q.nvfp4_bf16_linear(x, w, out=torch.empty(4, 40, dtype=BF, device=DEV)), ValueError),
            (lambda: q.nvfp4_bf16_linear(x, w, activation=9), RuntimeError),
            (lambda: q.nvfp4_bf16_linear(x, w3, ends=ends.long()), ValueError),
            (lambda: q.nvfp4_bf16_linear_backward(x, x[:, :32], q.ACT_SILU), ValueError),
            (lambda: q.nvfp4_bf16_linear_backward(x40, x40, q.ACT_SILU, workspace=torch.empty(16, dtype=torch.uint8, device=DEV)), ValueError)):
        with pytest.raises(error):
            call()
