"""Dispatch, combine and their gradients against plain sums in 64 bits: types,
one token to many, empty slots, pitches, places out of range, rows that nobody
names, far offsets.

Tolerances: a sum of k products in fp32, each rounding 2^-24 of the sum of
sizes (k + 1 of them at most), then half a step of the output's type; the dot
products' lanes add cols / 64 terms each, in waves and between them below cols / 64 + 16 steps."""
import pytest
import torch

import quantize_precision_gemm_amd as q

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def rng(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(seed, *shape):
    return torch.randn(shape, generator=rng(seed), device=DEV)


def places(seed, T, k, empty=0.2):
    """Every slot a row of its own, in no order; some none (-1)."""
    rows = torch.randperm(T * k, generator=rng(seed), device=DEV).int().view(T, k)
    return torch.where(torch.rand(T, k, generator=rng(seed + 1), device=DEV) < empty, -1, rows)


def pitched(t, more):
    """The same values, rows further apart."""
    wide = torch.full((t.shape[0], t.shape[1] + more), 3.0, dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


CASES = [(1, 1, 8), (1, 8, 5120), (2, 3, 64), (7, 8, 2048), (65, 2, 512), (33, 9, 520), (100, 6, 2568), (129, 4, 1024), (17, 64, 136),
         (5, 5, 9000), (3, 2, 16392), (1000, 1, 72)]


@pytest.mark.parametrize("T,k,cols", CASES)
@pytest.mark.parametrize("more", [0, 24])
def test_dispatch(T, k, cols, more):
    x = pitched(randn(1, T, cols).bfloat16(), more)
    rows = places(T, T, k)
    out = pitched(torch.full((T * k, cols), -5.0, dtype=torch.bfloat16, device=DEV), more)
    want = out.clone()
    got = q.nvfp4_dispatch(x, rows, out=out)
    there = rows >= 0
    want[rows[there].long()] = x[torch.arange(T, device=DEV)[:, None].expand(T, k)[there]]
    assert got is out and torch.equal(got, want)
    if more:
        assert (out._base[:, cols:] == 3).all()
    new = q.nvfp4_dispatch(x, rows)
    assert new.shape == (T * k, cols) and torch.equal(new[rows[there].long()], want[rows[there].long()])


@pytest.mark.parametrize("T,k,cols", CASES)
@pytest.mark.parametrize("o_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("y_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("weighted,residual", [(True, True), (False, False), (True, False)])
def test_combine(T, k, cols, o_dtype, y_dtype, weighted, residual):
    more = 8 if T % 2 else 0
    o = pitched(randn(2, T * k, cols).to(o_dtype), more)
    rows = places(T, T, k)
    w = torch.rand(T, k, generator=rng(3), device=DEV) if weighted else None
    r = pitched(randn(4, T, cols).to(y_dtype), more) if residual else None
    got = q.nvfp4_combine(o, rows, w, r, out_dtype=y_dtype)
    parts = o.double()[rows.clamp(min=0).long()] * (rows >= 0)[..., None]
    if weighted:
        parts = parts * w.double()[..., None]
    want, size = parts.sum(1), parts.abs().sum(1)
    if residual:
        want, size = want + r.double(), size + r.double().abs()
    assert ((got.double() - want).abs() <= (k + 1) * 2.0 ** -24 * size + HALF[y_dtype] * want.abs() * 1.001 + 2.0 ** -140).all()
    if residual:  # in place
        assert torch.equal(q.nvfp4_combine(o, rows, w, r, out=r), got)


@pytest.mark.parametrize("T,k,cols", CASES)
@pytest.mark.parametrize("dy_dtype,o_dtype", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.bfloat16),
                                              (torch.bfloat16, torch.float32), (torch.float32, torch.float32)])
def test_combine_backward(T, k, cols, dy_dtype, o_dtype):
    more = 16 if T % 2 else 0
    dy, o = pitched(randn(5, T, cols).to(dy_dtype), more), pitched(randn(6, T * k, cols).to(o_dtype), more)
    rows, w = places(T, T, k), torch.randn(T, k, generator=rng(7), device=DEV)
    out = torch.full((T * k, cols), -5.0, dtype=torch.bfloat16, device=DEV)
    got, dw = q.nvfp4_combine_backward(dy, o, rows, w, out=out)
    there = rows >= 0
    want = torch.full((T * k, cols), -5.0, dtype=torch.float64, device=DEV)
    scaled = dy.double()[:, None] * w.double()[..., None]
    want[rows[there].long()] = scaled[there]
    assert ((got.double() - want).abs() <= (2.0 ** -8 * 1.001 + 2.0 ** -24) * want.abs()).all()
    parts = dy.double()[:, None] * o.double()[rows.clamp(min=0).long()] * there[..., None]
    steps = cols / 64 + 16
    assert ((dw.double() - parts.sum(2)).abs() <= steps * 2.0 ** -24 * parts.abs().sum(2)).all()
    assert (dw[~there] == 0).all()
    # the gradients are those of combine: along a direction, its (linear) difference
    d = randn(8, T * k, cols).to(o_dtype)
    slope = (dy.double() * ((d.double()[rows.clamp(min=0).long()] * there[..., None]) * w.double()[..., None]).sum(1)).sum()
    named = torch.zeros(T * k, 1, dtype=torch.float64, device=DEV)
    named[rows[there].long()] = 1.0
    along = (got.double() * d.double() * named).sum()
    assert abs(along - slope) <= 2.0 ** -7 * (got.double() * d.double() * named).abs().sum() + 1e-30


def test_places_out_of_range_are_nobody():
    T, k, cols = 6, 3, 64
    x, o = randn(1, T, cols).bfloat16(), randn(2, 10, cols)
    rows = torch.tensor([[0, -1, 10], [9, 1 << 30, -(1 << 31)], [3, 2, -7], [1, 11, 4], [5, 6, 7], [8, 100, 12]], dtype=torch.int32,
                        device=DEV)
    out = torch.full((10, cols), 2.0, dtype=torch.bfloat16, device=DEV)
    q.nvfp4_dispatch(x, rows, out=out)
    there = (rows >= 0) & (rows < 10)
    want = torch.full_like(out, 2.0)
    want[rows[there].long()] = x[torch.arange(T, device=DEV)[:, None].expand(T, k)[there]]
    assert torch.equal(out, want)
    y = q.nvfp4_combine(o, rows, None, out_dtype=torch.float32)
    ref = (o[torch.where(there, rows, 0).long()].double() * there[..., None]).sum(1)
    assert torch.allclose(y.double(), ref, rtol=0, atol=1e-6)
    d, dw = q.nvfp4_combine_backward(y, o, rows, torch.ones(T, k, device=DEV))
    assert (dw[~there] == 0).all() and d.shape == (10, cols)


def test_not_finite():
    """A row that is not finite shows in its tokens alone; a weight that is not a number shows, on an empty slot too."""
    o = randn(1, 8, 64)
    o[2, 5], o[3, 6] = torch.inf, torch.nan
    rows = torch.tensor([[0, 1], [2, -1], [3, 4], [5, -1]], dtype=torch.int32, device=DEV)
    w = torch.tensor([[0.5, 0.5], [1.0, 0.0], [0.3, 0.7], [1.0, torch.nan]], device=DEV)
    y = q.nvfp4_combine(o, rows, w, out_dtype=torch.float32)
    assert torch.isfinite(y[0]).all() and torch.isinf(y[1, 5]) and torch.isfinite(y[1, :5]).all()
    assert torch.isnan(y[2, 6]) and torch.isfinite(y[2, 7:]).all() and torch.isnan(y[3]).all()


def test_empty():
    none = torch.empty(0, 2, dtype=torch.int32, device=DEV)
    assert q.nvfp4_dispatch(torch.empty(0, 64, dtype=torch.bfloat16, device=DEV), none).shape == (0, 64)
    assert q.nvfp4_combine(torch.empty(0, 64, device=DEV), none).shape == (0, 64)
    nobody = torch.full((3, 2), -1, dtype=torch.int32, device=DEV)
    r = randn(1, 3, 64).bfloat16()
    assert torch.equal(q.nvfp4_combine(torch.empty(0, 64, device=DEV), nobody, residual=r), r)
    d, dw = q.nvfp4_combine_backward(r, torch.empty(0, 64, device=DEV), nobody, torch.ones(3, 2, device=DEV))
    assert d.shape == (0, 64) and (dw == 0).all()
    x = torch.empty(3, 0, dtype=torch.bfloat16, device=DEV)
    assert q.nvfp4_combine(torch.empty(6, 0, device=DEV), nobody).shape == (3, 0)
    assert (q.nvfp4_combine_backward(x, torch.empty(6, 0, device=DEV), nobody, torch.ones(3, 2, device=DEV))[1] == 0).all()


def test_offsets_past_32_bits():
    """Rows whose bytes and elements lie beyond 2^32."""
    cols, R = 65536, 70000  # 4.6e9 elements, 9.2e9 bytes
    out = torch.empty(R, cols, dtype=torch.bfloat16, device=DEV)
    x = randn(1, 3, cols).bfloat16()
    rows = torch.tensor([[R - 1, 0], [R - 2, 40000], [65537, 12]], dtype=torch.int32, device=DEV)
    q.nvfp4_dispatch(x, rows, out=out)
    for t in range(3):
        for j in range(2):
            assert torch.equal(out[rows[t, j]], x[t])
    assert torch.equal(q.nvfp4_combine(out, rows, torch.full((3, 2), 0.5, device=DEV)), x)
    q.nvfp4_combine_backward(x, out, rows, torch.full((3, 2), 2.0, device=DEV), out=out)  # (each place read, then written)
    assert torch.equal(out[R - 1], 2 * x[0]) and torch.equal(out[65537], 2 * x[2])


def test_refusals():
    x, rows = randn(1, 4, 64).bfloat16(), places(1, 4, 2)
    with pytest.raises(TypeError):
        q.nvfp4_dispatch(x.float(), rows)
    with pytest.raises(TypeError):
        q.nvfp4_dispatch(x, rows.long())
    with pytest.raises(ValueError):
        q.nvfp4_dispatch(x, rows[:3])
    with pytest.raises(ValueError):
        q.nvfp4_dispatch(x, rows, out=torch.empty(8, 72, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ValueError):
        q.nvfp4_dispatch(x.t(), places(1, 64, 2))
    with pytest.raises(ValueError):
        q.nvfp4_combine(x, rows.t())
    with pytest.raises(TypeError):
        q.nvfp4_combine(x, rows, residual=torch.zeros(4, 64, device=DEV))
    with pytest.raises(TypeError):
        q.nvfp4_combine(x, rows, torch.ones(4, 2, dtype=torch.float64, device=DEV))
    with pytest.raises(RuntimeError):
        q.nvfp4_combine(x[:, :60], rows)
    with pytest.raises(RuntimeError):
        q.nvfp4_combine(torch.empty(9, 68, dtype=torch.bfloat16, device=DEV)[1:, :64], rows)
    with pytest.raises(ValueError):
        q.nvfp4_combine_backward(x, x, rows, torch.ones(4, 3, device=DEV))
    with pytest.raises(ValueError):
        q.nvfp4_combine_backward(x, x[:, :32], rows, torch.ones(4, 2, device=DEV))
