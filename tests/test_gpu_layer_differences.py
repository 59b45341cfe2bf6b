"""Gradients against differences of what they are gradients of: dispatch and
combine called at shifted inputs (whole numbers, so that both sides are exact and have
to be equal), and a block of experts whose loss is computed in 64 bits at
shifted inputs, the routing held."""
import pytest
import torch

import quantize_precision_gemm_amd as q
from quantize_precision_gemm_amd.step import TrainingStep
from tests.test_gpu_expert_block import ACTS, FAR, block_of
from tests.test_gpu_move_rows import places, rng

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def whole(seed, *shape, most=4):
    return torch.randint(-most, most + 1, shape, generator=rng(seed), device=DEV).float()


# Sums of at most 8 products of 4 x 1 and a residual, and dot products of 16392 at most: below 2^24, exact in fp32.
# Weights are sixteenths: their products with whole numbers up to 4 have 7 bits, exact in bf16.
@pytest.mark.parametrize("T,k,cols", [(1, 1, 8), (7, 8, 2048), (65, 2, 512), (33, 5, 520), (100, 6, 2568), (3, 2, 16392)])
@pytest.mark.parametrize("o_dtype", [torch.bfloat16, torch.float32])
def test_combine(T, k, cols, o_dtype):
    rows = places(T, T, k)
    o, d_o = whole(1, T * k, cols), whole(2, T * k, cols)
    w, d_w = whole(3, T, k, most=8) / 16, whole(4, T, k, most=8) / 16
    dy, r = whole(5, T, cols), whole(6, T, cols)

    def loss(o, w):
        y = q.nvfp4_combine(o.to(o_dtype), rows, w, r, out_dtype=torch.float32)
        return (y.double() * dy.double()).sum()
    grad_o, grad_w = q.nvfp4_combine_backward(dy, o.to(o_dtype), rows, w, out=torch.zeros(T * k, cols, dtype=torch.bfloat16, device=DEV))
    assert (grad_o.double() * d_o.double()).sum() == loss(o + d_o, w) - loss(o, w)
    assert (grad_w.double() * d_w.double()).sum() == loss(o, w + d_w) - loss(o, w)


@pytest.mark.parametrize("T,k,cols", [(1, 1, 8), (7, 8, 2048), (33, 5, 520), (3, 2, 16392)])
def test_dispatch(T, k, cols):
    rows = places(T, T, k)
    x, d = whole(1, T, cols), whole(2, T, cols)
    g = whole(3, T * k, cols)

    def loss(x):
        out = q.nvfp4_dispatch(x.bfloat16(), rows, out=torch.zeros(T * k, cols, dtype=torch.bfloat16, device=DEV))
        return (out.double() * g.double()).sum()
    grad = q.nvfp4_combine(g, rows, out_dtype=torch.float32)
    assert (grad.double() * d.double()).sum() == loss(x + d) - loss(x)


def block_loss(b, x, norm_weight, router, w1, b1, w2):
    """<y, dy> in 64 bits, token by token and slot by slot, with the block's choices."""
    h = x + b.residual.double()
    n = h / torch.sqrt(h.square().mean(1, keepdim=True) + b.eps) * norm_weight
    logits = n @ router.t()
    experts = b.routing.experts.long()
    s = torch.sigmoid(logits) if b.route_args["score"] == q.SIGMOID else torch.softmax(logits, 1)
    w = s.gather(1, experts)
    if b.route_args["renormalise"]:
        w = w / w.sum(1, keepdim=True)
    y = h.clone()
    for e in range(b.E):
        t, j = torch.nonzero(experts == e, as_tuple=True)
        a = ACTS[b.activation](n[t] @ w1[e].t() + b1[e])
        y.index_add_(0, t, b.route_args["scale"] * w[t, j, None] * (a @ w2[e].t()))
    return (y * b.dy.double()).sum()


@pytest.mark.parametrize("T,H,E,F,k,how", [
    (37, 128, 8, 72, 3, dict(score=q.SIGMOID, activation=q.ACT_SILU)), (300, 64, 24, 64, 8, dict(renormalise=False)),
    (200, 256, 16, 136, 4, dict(score=q.SIGMOID, scale=2.5, activation=q.ACT_GELU))])
def test_block(T, H, E, F, k, how):
    """Along each gradient itself: the loss changes by its length.  A gradient's
    relative norm is off by at most FAR (test_gpu_expert_block.py); a quotient of steps of
    2^-12 of an input's norm by some 2^-24 of the loss's curvature, below 2^-10."""
    b = block_of(T, H, E, F, k, **how)
    TrainingStep(torch, [b], torch.device(DEV)).run()
    torch.cuda.synchronize()
    at = {name: getattr(b, name).double() for name in ("x", "norm_weight", "router", "w1", "b1", "w2")}
    grads = dict(x=b.dx, norm_weight=b.dnorm, router=b.drouter[0], w1=b.dw1, b1=b.db1, w2=b.dw2)
    for name, grad in grads.items():
        grad = grad.double()
        length = grad.norm()
        step = 2.0 ** -12 * at[name].norm()
        d = grad / length * step
        slope = (block_loss(b, **dict(at, **{name: at[name] + d})) - block_loss(b, **dict(at, **{name: at[name] - d}))) / (2 * step)
        assert abs(slope / length - 1) <= FAR * 1.04 + 2.0 ** -10, (name, (slope / length).item())
