"""Routing against its definition in 64 bits (numpy, one token at a time where
choices are made): experts, places and ends have to be equal, weights and scores
within roundings.  Ties, near ties that fp32 cannot tell apart, masked and
padded tokens, logits and biases that are not finite, every size of the
kernels' variants; the gradient against the formula's and against differences.

Tolerances, in units of 2^-24 of the value: a score is e^x (x rounded by |x| / 2
units of an argument up to 30 away from the largest: 30; the exponential 4), a sum
of up to 1024 of them in at most 24 steps (24) and a quotient or two (4):
below 64 units, 2^-18."""
import numpy as np
import pytest
import torch

import quantize_precision_gemm_amd as q

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TOL = 2.0 ** -18


def scores_of(l, score):
    l = l.astype(np.float64)
    with np.errstate(over="ignore"):
        if score == q.SIGMOID:
            return 1.0 / (1.0 + np.exp(-l))
        top = l.max(1, keepdims=True)
        e = np.exp(l - np.where(np.isfinite(top), top, 0.0))
    total = e.sum(1, keepdims=True)
    return e / np.where(total > 0, total, 1.0)


def definition(logits, k, score, bias=None, groups=1, kept=None, renorm=True, scale=1.0):
    """(experts, weights, rows, ends, scores) of a float64 array of logits."""
    T, E = logits.shape
    kept = groups if kept is None else kept
    bad = ~(logits < np.inf).all(1)  # NaN or plus infinity somewhere
    l = np.where(np.isfinite(logits), logits, -np.inf)
    s = scores_of(l, score)
    c = s + (0.0 if bias is None else bias.astype(np.float64)[None])
    c = np.where(np.isfinite(l) & np.isfinite(c), c, -np.inf)
    experts = np.full((T, k), -1, dtype=np.int32)
    weights = np.zeros((T, k))
    for t in range(T):
        open_ = c[t] > -np.inf
        if kept < groups:
            value = np.full(groups, -np.inf)
            for g in range(groups):
                best = np.sort(c[t].reshape(groups, -1)[g])[::-1][:2]
                best = best[best > -np.inf]
                if len(best):
                    value[g] = best.sum()
            order = np.argsort(-value, kind="stable")[:kept]
            stays = np.zeros(groups, dtype=bool)
            stays[order] = True
            open_ &= np.repeat(stays, E // groups)
        by = np.where(open_, l[t] if bias is None else c[t], -np.inf)
        picked = [e for e in np.argsort(-by, kind="stable")[:k] if open_[e]]
        experts[t, :len(picked)] = picked
        w = s[t, picked]
        if renorm and len(picked):
            # as a softmax of logarithms, so that small scores do not vanish
            x = l[t, picked] if score == q.SOFTMAX else -np.logaddexp(0.0, -l[t, picked])
            w = np.exp(x - x.max())
            w = w / w.sum()
        weights[t, :len(picked)] = scale * w
    weights[bad] = np.nan
    s = np.where(bad[:, None], np.nan, s)
    flat = np.where(experts.reshape(-1) < 0, E, experts.reshape(-1))
    order = np.argsort(flat, kind="stable")
    rows = np.empty(T * k, dtype=np.int64)
    rows[order] = np.arange(T * k)
    rows = np.where(flat < E, rows, -1).reshape(T, k)
    ends = np.searchsorted(flat[order], np.arange(E), side="right")
    return experts, weights, rows, ends, s


def check(logits, k, score, bias=None, groups=1, kept=None, renorm=True, scale=1.0, **how):
    """logits: a device tensor, bias a device tensor or None."""
    want = definition(logits.double().cpu().numpy(), k, score, None if bias is None else bias.cpu().numpy(), groups, kept, renorm,
                      scale)
    r = q.nvfp4_route(logits, k, score, bias=bias, groups=groups, groups_kept=kept, renormalise=renorm, scale=scale,
                      with_scores=True, **how)
    np.testing.assert_array_equal(r.experts.cpu().numpy(), want[0])
    np.testing.assert_array_equal(r.rows.cpu().numpy(), want[2])
    np.testing.assert_array_equal(r.ends.cpu().numpy(), want[3])
    # (fp32 holds nothing below 2^-126 to full precision)
    np.testing.assert_allclose(r.weights.double().cpu().numpy(), want[1], rtol=TOL, atol=2.0 ** -126 * abs(scale))
    np.testing.assert_allclose(r.scores.double().cpu().numpy(), want[4], rtol=TOL, atol=2.0 ** -126)
    return r


def randn(seed, *shape, scale=1.5):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return scale * torch.randn(shape, generator=g, device=DEV)


SIZES = [(1, 1, 1), (1, 64, 8), (3, 2, 2), (16, 7, 3), (63, 16, 4), (64, 17, 16), (65, 32, 1), (100, 33, 2), (128, 64, 8), (200, 65, 6),
         (129, 100, 8), (70, 128, 10), (300, 129, 4), (65, 256, 8), (1000, 256, 8), (90, 257, 3), (17, 300, 5), (130, 512, 16),
         (40, 513, 8), (65, 1000, 9), (33, 1024, 16)]


@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("score", [q.SOFTMAX, q.SIGMOID])
@pytest.mark.parametrize("biased", [False, True])
def test_route(T, E, k, score, biased):
    seed = T * 10000 + E
    logits = randn(seed, T, E)
    bias = randn(seed + 1, E, scale=0.1) if biased else None
    check(logits, k, score, bias, renorm=(T + k) % 2 == 0, scale=2.5 if E % 2 else 1.0)
    check(logits.bfloat16(), k, score, bias)


@pytest.mark.parametrize("T,E,G,kept,k", [(1, 4, 2, 1, 2), (65, 8, 8, 3, 3), (64, 16, 4, 2, 6), (33, 60, 6, 2, 4), (100, 64, 8, 4, 8),
                                          (129, 96, 3, 2, 5), (70, 160, 8, 3, 6), (130, 256, 8, 4, 8), (20, 250, 2, 1, 8),
                                          (65, 512, 16, 5, 8), (9, 1024, 64, 3, 16), (9, 64, 64, 5, 5), (65, 128, 1, 1, 8)])
@pytest.mark.parametrize("score", [q.SOFTMAX, q.SIGMOID])
@pytest.mark.parametrize("biased", [False, True])
def test_groups(T, E, G, kept, k, score, biased):
    logits = randn(E + T, T, E)
    bias = randn(E, E, scale=0.1) if biased else None
    check(logits, k, score, bias, G, kept)
    check(logits.bfloat16(), k, score, bias, G, kept, renorm=False)


@pytest.mark.parametrize("T", [16384, 16385, 20011])
def test_many_chunks(T):
    """Counts summed by each workgroup (256 chunks), and by a kernel of their own."""
    logits = randn(T, T, 24)
    r = q.nvfp4_route(logits, 4, q.SOFTMAX)
    experts = torch.sort(logits, dim=1, descending=True, stable=True)[1][:, :4].int()
    assert torch.equal(r.experts, experts)
    flat = experts.flatten().long()
    order = flat.sort(dim=0, stable=True)[1]
    rows = torch.empty_like(order)
    rows[order] = torch.arange(4 * T, device=DEV)
    assert torch.equal(r.rows.flatten().long(), rows)
    assert torch.equal(r.ends.long(), torch.cumsum(torch.bincount(flat, minlength=24), 0))


@pytest.mark.parametrize("score", [q.SOFTMAX, q.SIGMOID])
@pytest.mark.parametrize("groups,kept", [(1, 1), (4, 2)])
@pytest.mark.parametrize("E", [16, 64, 256, 320])
def test_ties(E, groups, kept, score):
    """Equal logits (also +0 and -0), with no bias, a bias of zeros and one of equal steps: the lowest index first."""
    logits = torch.round(randn(E, 77, E)) * 0.5
    logits[3] = 0.0
    logits[4] = torch.where(torch.arange(E, device=DEV) % 2 == 0, -0.0, 0.0)
    bias = torch.round(randn(E + 1, E)) * 0.0625
    for b in (None, torch.zeros(E, device=DEV), bias):
        check(logits, 5, score, b, groups, kept)


@pytest.mark.parametrize("score", [q.SOFTMAX, q.SIGMOID])
@pytest.mark.parametrize("E", [32, 256, 400])
def test_choices_that_fp32_cannot_tell_apart(E, score):
    """Biases that make pairs of experts all but equal for a token: which of two
    comes first is decided by differences next to 2^-26 (a bias's own rounding)."""
    T = 96
    logits = randn(E + 5, T, E).double()
    s = scores_of(logits.float().cpu().numpy(), score)
    found = 0
    for t in range(0, T, 3):
        bias = np.zeros(E, dtype=np.float32)
        a, b = t % E, (t * 7 + 1) % E
        if a == b:
            continue
        bias[a] = 0.75
        bias[b] = np.float32(s[t, a] + 0.75 - s[t, b])
        gap = abs((s[t, a] + 0.75) - (s[t, b] + float(bias[b])))
        found += 0 < gap < 2.0 ** -23
        check(logits[t:t + 1].float(), 2, score, torch.tensor(bias, device=DEV))
    assert found > 20
    # the same for groups: two whose best pairs add up to nearly the same
    bias = np.zeros(E, dtype=np.float32)
    G, per = 2, E // 2
    for t in range(0, T, 3):
        bias[:] = 0
        first = np.sort(s[t, :per])[::-1][:2].sum()
        at = per + np.argsort(-s[t, per:])[:2]
        bias[at[0]] = np.float32(first - s[t, at].sum())
        check(logits[t:t + 1].float(), 3, score, torch.tensor(bias, device=DEV), G, 1)


@pytest.mark.parametrize("score", [q.SOFTMAX, q.SIGMOID])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("groups,kept", [(1, 1), (4, 3)])
def test_masked_and_not_finite(groups, kept, score, biased):
    T, E, k = 140, 32, 6
    logits = randn(9, T, E)
    logits[0] = -torch.inf                       # padded
    logits[1, 3:] = -torch.inf                   # three left
    logits[2, :] = -torch.inf
    logits[2, 17] = -80.0                        # one, far down
    logits[3, 5] = torch.nan
    logits[4, 6] = torch.inf
    logits[5] = torch.nan
    logits[6, ::2] = torch.finfo(torch.float32).min  # the type's lowest value is a value
    logits[7] = torch.finfo(torch.float32).min
    logits[8, :20] = -torch.inf                  # whole groups
    logits[70:80] = -torch.inf
    logits[-1] = -torch.inf
    bias = None
    if biased:
        bias = randn(3, E, scale=0.1)
        bias[1], bias[2], bias[3] = -torch.inf, torch.inf, torch.nan
    for renorm in (True, False):
        r = check(logits, k, score, bias, groups, kept, renorm)
    used = int((r.rows >= 0).sum())
    assert used < T * k and int(r.ends[-1]) == used
    check(torch.full((70, E), -torch.inf, device=DEV), k, score, bias, groups, kept)


@pytest.mark.parametrize("E,k", [(8, 8), (20, 5), (256, 4)])
@pytest.mark.parametrize("score", [q.SOFTMAX, q.SIGMOID])
def test_values_far_apart(E, k, score):
    """Finite logits whose differences overflow, or pass what the fast comparison spans; biases of any size."""
    big = torch.finfo(torch.float32).max
    logits = randn(1, 12, E)
    logits[0, :3] = torch.tensor([big, -big, -big], device=DEV)
    logits[1] = -big
    logits[1, 2] = big
    logits[2] = torch.linspace(-big, big, E, device=DEV)
    logits[3] = 1e-38 * logits[3]
    logits[4, 1:] -= 40.0
    logits[5, k - 1:] -= 1e6
    check(logits, k, score)
    for size in (1e-30, 5.0, 1e8, 1e38, 3e38):
        check(logits, k, score, size * randn(2, E, scale=0.5).clamp(-1, 1))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,pitch,offset", [(64, 68, 0), (64, 67, 0), (64, 72, 3), (33, 33, 0), (256, 261, 1), (300, 512, 0)])
def test_strides_and_alignment(E, pitch, offset, dtype):
    buf = randn(E, 90 * pitch + offset).to(dtype)
    logits = buf[offset:offset + 90 * pitch].view(90, pitch)[:, :E]
    check(logits, 4, q.SIGMOID, randn(2, E, scale=0.1))


def test_no_tokens_and_no_places():
    r = q.nvfp4_route(torch.empty(0, 12, device=DEV), 3)
    assert r.experts.shape == (0, 3) and torch.equal(r.ends, torch.zeros(12, dtype=torch.int32, device=DEV))
    logits = randn(1, 70, 12)
    want = q.nvfp4_route(logits, 3)
    experts, weights = torch.empty(70, 3, dtype=torch.int32, device=DEV), torch.empty(70, 3, device=DEV)
    st = q.load_library().nvfp4_route(logits.data_ptr(), 1, 12, 70, 12, 3, None, 1, 1, 0, 1, 1.0, experts.data_ptr(),
                                      weights.data_ptr(), None, None, None, None, 0, None)
    torch.cuda.synchronize()
    assert st == 0 and torch.equal(experts, want.experts) and torch.equal(weights, want.weights)
    g = q.nvfp4_route_backward(torch.empty(0, 12, device=DEV), torch.empty(0, 3, dtype=torch.int32, device=DEV),
                               torch.empty(0, 3, device=DEV))
    assert g.shape == (0, 12)


def test_buffers_kept_and_refused():
    logits = randn(4, 300, 40)
    plan = q.Routing.empty(300, 40, 4, torch.device(DEV))
    first = q.nvfp4_route(logits, 4, out=plan)
    assert first is plan
    kept = [t.clone() for t in (plan.experts, plan.weights, plan.rows, plan.ends)]
    q.nvfp4_route(randn(5, 300, 40), 4, out=plan)
    q.nvfp4_route(logits, 4, out=plan)
    for a, b in zip(kept, (plan.experts, plan.weights, plan.rows, plan.ends)):
        assert torch.equal(a, b)
    with pytest.raises(ValueError):
        q.nvfp4_route(randn(5, 301, 40), 4, out=plan)
    with pytest.raises(ValueError):
        q.nvfp4_route(logits, 4, out=plan, with_scores=True)
    with pytest.raises(ValueError):
        q.nvfp4_route(logits, 4, out=q.Routing(plan.experts, plan.weights, plan.rows, plan.ends,
                                               workspace=plan.workspace[:64]))
    with pytest.raises(ValueError):
        q.nvfp4_route(logits, 4, bias=torch.zeros(41, device=DEV))
    with pytest.raises(TypeError):
        q.nvfp4_route(logits.half(), 4)
    with pytest.raises(ValueError):
        q.nvfp4_route(logits.t(), 4)
    with pytest.raises(RuntimeError):
        q.nvfp4_route(logits, 17)
    with pytest.raises(RuntimeError):
        q.nvfp4_route(logits, 4, groups=7)
    torch.cuda.synchronize()


# ---- gradients ----

def weights_of(l, experts, score, renorm, scale):
    """The chosen weights as a differentiable function of float64 logits (T x E)."""
    there = experts >= 0
    at = experts.clamp(min=0).long()
    if renorm:
        x = torch.nn.functional.logsigmoid(l) if score == q.SIGMOID else l
        x = x.gather(1, at).masked_fill(~there, -torch.inf)
        none = ~there.any(1, keepdim=True)
        return scale * torch.softmax(x.masked_fill(none, 0.0), 1) * there
    s = torch.sigmoid(l) if score == q.SIGMOID else torch.softmax(l, 1)
    return scale * s.gather(1, at) * there


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 8, 3), (64, 16, 16), (33, 60, 6), (100, 128, 8), (50, 256, 8), (31, 300, 5), (9, 1024, 16)])
@pytest.mark.parametrize("score", [q.SOFTMAX, q.SIGMOID])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("with_scores", [False, True])
def test_backward(T, E, k, score, renorm, with_scores):
    """Tolerance: a gradient is a factor of at most 64 units of 2^-24 (as above) off,
    and a difference of terms whose sizes the bound adds up."""
    logits = randn(T + E, T, E)
    experts = q.nvfp4_route(logits, k, score, bias=randn(E, E, scale=0.1)).experts
    if T > 3:
        experts[2] = -1
        experts[3, k // 2:] = -1
    dw, ds = randn(7, T, k), randn(8, T, E) if with_scores else None
    got = q.nvfp4_route_backward(logits, experts, dw, score, renorm, 1.5, ds).double().cpu()
    l = logits.double().cpu().requires_grad_()
    w = weights_of(l, experts.cpu(), score, renorm, 1.5)
    s = torch.sigmoid(l) if score == q.SIGMOID else torch.softmax(l, 1)
    total = (w * dw.double().cpu()).sum() + ((s * ds.double().cpu()).sum() if with_scores else 0.0)
    want, = torch.autograd.grad(total, l)
    p = torch.zeros(T, E, dtype=torch.float64).scatter_add_(1, experts.cpu().clamp(min=0).long(), w.detach())
    size = 1.5 * dw.abs().max().double().cpu() * (p + s.detach()) * 2 + (2 * ds.abs().max().double().cpu() * s.detach() if with_scores else 0.0)
    assert ((got - want).abs() <= TOL * size + 2.0 ** -126).all()
    # a difference quotient along one direction (float64): the same number
    d = torch.randn(T, E, dtype=torch.float64, generator=torch.Generator().manual_seed(3))

    def value(x):
        x = l.detach() + x * d
        y = (weights_of(x, experts.cpu(), score, renorm, 1.5) * dw.double().cpu()).sum()
        x = torch.sigmoid(x) if score == q.SIGMOID else torch.softmax(x, 1)
        return y + ((x * ds.double().cpu()).sum() if with_scores else 0.0)
    h = 1e-5
    slope = (value(h) - value(-h)) / (2 * h)
    # the quotient is off by h^2 / 6 of a third derivative: below 1e-9 of the sum of sizes
    assert abs((got * d).sum() - slope) <= (TOL + 1e-8) * (size * d.abs()).sum() + 1e-12
    half = q.nvfp4_route_backward(logits, experts, dw, score, renorm, 1.5, ds, out_dtype=torch.bfloat16).double().cpu()
    assert ((half - want).abs() <= TOL * size + 2.0 ** -8 * want.abs() * 1.01 + 2.0 ** -126).all()


def test_backward_masked_repeated_and_strided():
    T, E = 40, 48
    logits = randn(1, T, E)
    logits[:, 10:20] = -torch.inf
    logits[5] = -torch.inf
    experts = torch.randint(0, 10, (T, 4), generator=torch.Generator().manual_seed(1)).int().to(DEV)  # some twice in a row
    experts[5] = -1
    experts[6, 1], experts[6, 2] = E, 1 << 30  # out of range: no part
    dw = randn(2, T, 4)
    buf = torch.full((T, E + 5), 7.0, device=DEV)
    got = q.nvfp4_route_backward(logits, experts, dw, q.SOFTMAX, False, out=buf[:, 1:E + 1])
    l = logits.double().cpu().masked_fill(logits.cpu() == -torch.inf, -1e300).requires_grad_()
    e = torch.where((experts < 0) | (experts >= E), -1, experts).cpu()
    w = weights_of(l, e, q.SOFTMAX, False, 1.0)
    want, = torch.autograd.grad((w * dw.double().cpu()).sum(), l)
    want[5] = 0.0
    np.testing.assert_allclose(got.double().cpu().numpy(), want.numpy(), atol=8 * TOL * float(dw.abs().max()), rtol=0)
    assert (got[:, 10:20] == 0).all() and (got[5] == 0).all()
    assert (buf[:, 0] == 7).all() and (buf[:, E + 1:] == 7).all()
