"""Norm, router, dispatch, products, combine and all their gradients together,
as the training-step driver runs them (BF16ExpertBlock): against a plain block in
64 bits with its gradients, captured and replayed, on other streams, and the
example that trains one.

Tolerances: relative norms.  A result passes through at most 8 roundings to bf16
(n, the sums before the activation, act, o, y; back do, dact, dpre, drows, dx),
each at most 2^-8 of a value; the maps between them are well conditioned, so
their sum, 2^-5, bounds the relative norm."""
import os
import sys

import pytest
import torch

import quantize_precision_gemm_amd as q
from quantize_precision_gemm_amd.step import BF16ExpertBlock, BF16Linear, TrainingStep
from tests.gpu_util import ROOT

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
FAR = 2.0 ** -5


def rng(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def inputs(seed, T, H):
    g = rng(seed)
    return [torch.randn(T, H, generator=g, device=DEV).bfloat16() for _ in range(3)]


def block_of(T, H, E, F, k, seed=0, **how):
    g = rng(seed)

    def randn(*s):
        return torch.randn(s, generator=g, device=DEV)
    x, residual, dy = inputs(seed + 1, T, H)
    return BF16ExpertBlock(q, torch, x, residual, dy, 1 + 0.1 * randn(H), (randn(E, H) * H ** -0.5).bfloat16(),
                           (randn(E, F, H) * H ** -0.5).bfloat16(), 0.1 * randn(E, F), (randn(E, H, F) * F ** -0.5).bfloat16(), k, **how)


OUTPUTS = ("y", "h", "dx", "dnorm", "drouter", "dw1", "db1", "dw2")
ACTS = {q.ACT_RELU2: lambda z: torch.relu(z) ** 2, q.ACT_SILU: torch.nn.functional.silu,
        q.ACT_GELU: lambda z: torch.nn.functional.gelu(z, approximate="tanh")}


def reference(b):
    """The block in 64 bits with its gradients; which experts a token goes to is taken from the block."""
    x, norm, router, w1, b1, w2 = (t.double().requires_grad_() for t in (b.x, b.norm_weight, b.router, b.w1, b.b1, b.w2))
    h = x + b.residual.double()
    n = h / torch.sqrt(h.square().mean(1, keepdim=True) + b.eps) * norm
    logits = n @ router.t()
    experts = b.routing.experts.long()
    chosen = logits.gather(1, experts)
    if b.route_args["score"] == q.SIGMOID:
        s = torch.sigmoid(chosen)
        w = s / s.sum(1, keepdim=True) if b.route_args["renormalise"] else s
    else:
        w = torch.softmax(chosen, 1) if b.route_args["renormalise"] else torch.softmax(logits, 1).gather(1, experts)
    w = w * b.route_args["scale"]
    y = h
    for j in range(b.k):
        e = experts[:, j]
        z = torch.matmul(w1[e], n[:, :, None])[:, :, 0] + b1[e]
        o = torch.matmul(w2[e], ACTS[b.activation](z)[:, :, None])[:, :, 0]
        y = y + w[:, j:j + 1] * o
    grads = torch.autograd.grad((y * b.dy.double()).sum(), (x, norm, router, w1, b1, w2))
    dx, dnorm, drouter, dw1, db1, dw2 = grads
    return dict(y=y.detach(), h=h.detach(), dx=dx, dnorm=dnorm, drouter=drouter[None], dw1=dw1, db1=db1, dw2=dw2)


def distance(a, b):
    return ((a.double() - b.double()).norm() / b.double().norm()).item()


@pytest.mark.parametrize("T,H,E,F,k,how", [
    (1, 64, 8, 128, 2, {}), (37, 128, 8, 72, 3, dict(score=q.SIGMOID, activation=q.ACT_SILU)),
    (200, 256, 16, 136, 4, dict(score=q.SIGMOID, groups=4, groups_kept=2, scale=2.5, activation=q.ACT_GELU)),
    (300, 64, 24, 64, 8, dict(renormalise=False)), (130, 512, 8, 256, 1, dict(renormalise=False, score=q.SIGMOID))])
def test_block(T, H, E, F, k, how):
    how = dict(how)
    if how.get("groups"):
        how["choice_bias"] = 0.05 * torch.randn(E, generator=rng(5), device=DEV)
    b = block_of(T, H, E, F, k, **how)
    TrainingStep(torch, [b], torch.device(DEV)).run()
    torch.cuda.synchronize()
    assert int(b.routing.ends[-1]) == T * k
    want = reference(b)
    for name in OUTPUTS:
        got = getattr(b, name)
        assert distance(got, want[name]) <= FAR, name
    # the gradient against a difference of the loss along one direction of w2 (the block is linear in it)
    d = torch.randn(b.w2.shape, generator=rng(9), device=DEV).double()
    slope = (want["dw2"] * d).sum()
    assert abs((b.dw2.double() * d).sum() - slope) <= FAR * want["dw2"].norm() * d.norm()


@pytest.mark.parametrize("serial", [False, True])
def test_beside_another_layer(serial):
    """In one training step with a plain layer: the same bits as its operations one by one."""
    b = block_of(300, 128, 8, 136, 2)
    x, w, dy = inputs(3, 304, 128)
    dense = BF16Linear(q, torch, x, w[:136].contiguous(), inputs(4, 304, 136)[0])
    TrainingStep(torch, [dense, b], torch.device(DEV), serial_gemms=serial).run()
    torch.cuda.synchronize()
    got = {name: getattr(b, name).clone() for name in OUTPUTS}
    for name in OUTPUTS:
        getattr(b, name).zero_()
    for _, op in b.forward_ops() + b.backward_shared_ops() + b.dgrad_ops() + b.wgrad_ops():
        op()
    torch.cuda.synchronize()
    for name in OUTPUTS:
        assert torch.equal(got[name], getattr(b, name)), name


@pytest.mark.parametrize("T", [40, 700])
def test_captured_and_replayed(T):
    """A step in a graph: replays on new inputs, other work between them, give the bits of eager steps; two graphs beside each other
    with buffers of their own."""
    blocks = [block_of(T, 128, 8, 136, 2, seed=s, score=q.SIGMOID, activation=q.ACT_SILU) for s in (1, 50)]
    steps = [TrainingStep(torch, [b], torch.device(DEV)) for b in blocks]
    for s in steps:
        s.run()
    torch.cuda.synchronize()
    graphs = []
    for s in steps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.run()
        graphs.append(g)
    for turn in range(4):
        want = []
        for b, s in zip(blocks, steps):
            for t, v in zip((b.x, b.residual, b.dy), inputs(100 + turn, T, 128)):
                t.copy_(v)
            s.run()
            torch.cuda.synchronize()
            want.append({name: getattr(b, name).clone() for name in OUTPUTS})
            for name in OUTPUTS:
                getattr(b, name).zero_()
        for g in graphs:
            g.replay()
        torch.randn(1000, 1000, device=DEV) @ torch.randn(1000, 1000, device=DEV)
        torch.cuda.synchronize()
        for b, w in zip(blocks, want):
            for name in OUTPUTS:
                assert torch.equal(getattr(b, name), w[name]), (turn, name)


def test_padded_tokens():
    """Tokens whose logits are all minus infinity go nowhere: their rows stay out of every sum, their outputs are the residual."""
    T, H, E, F, k = 90, 64, 8, 72, 2
    b = block_of(T, H, E, F, k)
    pad = torch.arange(T, device=DEV) % 3 == 0
    for t in (b.rows, b.do, b.dpre, b.act, b.pre):  # what lies behind the last expert's rows must not matter
        t.fill_(float("nan"))
    ops = dict(b.forward_ops() + b.backward_shared_ops() + b.dgrad_ops() + b.wgrad_ops())
    for name, op in ops.items():
        op()
        if name == "block_router":
            b.logits[pad] = -torch.inf
    torch.cuda.synchronize()
    assert int(b.routing.ends[-1]) == int((~pad).sum()) * k
    assert (b.routing.rows[pad] == -1).all() and torch.equal(b.y[pad], b.h[pad])
    for name in OUTPUTS:
        assert torch.isfinite(getattr(b, name)).all(), name
    full = {name: getattr(b, name).clone() for name in OUTPUTS}
    small = BF16ExpertBlock(q, torch, *(t[~pad].contiguous() for t in (b.x, b.residual, b.dy)), b.norm_weight, b.router, b.w1, b.b1, b.w2, k)
    TrainingStep(torch, [small], torch.device(DEV)).run()
    torch.cuda.synchronize()
    assert distance(full["y"][~pad], small.y) <= 2.0 ** -7 and distance(full["dx"][~pad], small.dx) <= FAR
    for name in ("dw1", "db1", "dw2", "drouter"):
        assert distance(full[name], getattr(small, name)) <= 2.0 ** -7, name


def calls():
    """One call of each operator, with inputs of its own; stream: where it runs."""
    T, E, k, H, F = 300, 16, 3, 136, 72
    logits = torch.randn(T, E, generator=rng(1), device=DEV)
    r = q.nvfp4_route(logits, k)
    x, residual, dy = inputs(2, T, H)
    o, w = torch.randn(T * k, H, generator=rng(3), device=DEV), torch.ones(H, device=DEV)
    w1, b1 = torch.randn(E, F, H, generator=rng(4), device=DEV).bfloat16(), torch.randn(E, F, generator=rng(5), device=DEV)
    xe = q.nvfp4_dispatch(x, r.rows)
    pre = torch.randn(T * k, F, generator=rng(6), device=DEV).bfloat16()

    def routed(stream):
        p = q.nvfp4_route(logits, k, with_scores=True, stream=stream)
        return [p.experts, p.weights, p.rows, p.ends, p.scores]

    x128, residual128 = x[:, :128].contiguous(), residual[:, :128].contiguous()  # (int8 rows come in sixteens)

    def int8(stream):
        y, h = q.nvfp4_rmsnorm_i8(x128, w[:128].contiguous(), residual=residual128, stream=stream)
        return [y.codes, y.scales, h]
    torch.cuda.synchronize()
    return {
        "route": routed,
        "route_backward": lambda s: [q.nvfp4_route_backward(logits, r.experts, r.weights, stream=s)],
        "dispatch": lambda s: [q.nvfp4_dispatch(x, r.rows, stream=s)],
        "combine": lambda s: [q.nvfp4_combine(o, r.rows, r.weights, residual=residual, stream=s)],
        "combine_backward": lambda s: list(q.nvfp4_combine_backward(dy, o, r.rows, r.weights, stream=s)),
        "rmsnorm": lambda s: list(q.nvfp4_rmsnorm(x, w, residual=residual, stream=s)),
        "rmsnorm_i8": int8,
        "rmsnorm_backward": lambda s: list(q.nvfp4_rmsnorm_backward(dy, x, w, dh=residual, stream=s)),
        "linear": lambda s: list(q.nvfp4_bf16_linear(xe, w1, ends=r.ends, bias=b1, activation=q.ACT_SILU, with_pre=True, stream=s)),
        "linear_backward": lambda s: list(q.nvfp4_bf16_linear_backward(pre, pre, q.ACT_SILU, ends=r.ends, stream=s)),
    }


@pytest.mark.parametrize("what", ["route", "route_backward", "dispatch", "combine", "combine_backward", "rmsnorm", "rmsnorm_i8",
                                  "rmsnorm_backward", "linear", "linear_backward"])
def test_outputs_on_another_stream(what):
    """Outputs and workspaces made for another stream are its own: memory freed on the current one, where work on
    it still waits, is not given to them."""
    call = calls()[what]
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    held = [torch.empty(t.numel() * t.element_size(), dtype=torch.uint8, device=DEV) for t in want]
    held += [torch.empty(n, dtype=torch.uint8, device=DEV) for n in (1 << 12, 1 << 16, 1 << 20)]
    torch.cuda._sleep(20_000_000)  # about 10 ms
    for t in held:
        t.fill_(255)
    del held, t
    got = call(side)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_inputs_dropped_before_another_stream_has_read_them():
    side = torch.cuda.Stream()
    x, residual, dy = inputs(2, 300, 136)
    w = torch.ones(136, device=DEV)
    logits = torch.randn(300, 16, generator=rng(1), device=DEV)
    r = q.nvfp4_route(logits, 3)
    want = [q.nvfp4_rmsnorm(x, w, residual=residual)[0], q.nvfp4_dispatch(x, r.rows), r.rows.clone(),
            q.nvfp4_combine(dy, r.rows[:100], r.weights[:100].contiguous())]
    torch.cuda.synchronize()
    for which in range(4):
        torch.cuda.empty_cache()
        tensors = [t.clone() for t in (x, residual, dy, w, logits, r.rows, r.weights)]
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        a, b, c, d, l, rows, weights = tensors
        got = (lambda: q.nvfp4_rmsnorm(a, d, residual=b, stream=side)[0], lambda: q.nvfp4_dispatch(a, rows, stream=side),
               lambda: q.nvfp4_route(l, 3, stream=side).rows,
               lambda: q.nvfp4_combine(c, rows[:100], weights[:100], stream=side))[which]()
        sizes = [t.numel() * t.element_size() for t in tensors]
        del a, b, c, d, l, rows, weights, tensors
        for n in sizes:
            torch.empty(n, dtype=torch.uint8, device=DEV).fill_(255)
        torch.cuda.synchronize()
        assert torch.equal(got, want[which]), which


def test_the_example_runs():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import expert_block
    losses, block, task = expert_block.train(steps=3, tokens=200, hidden=64, experts=8, inner=72)
    assert all(v == v for v in losses)
    x, residual, _ = task.batch(3)
    y, answers = expert_block.ask(block, x, residual, q.nvfp4_i8_quantize(task.randn(64, 64).bfloat16()))
    assert torch.isfinite(y).all() and answers.shape == (3, 64) and torch.isfinite(answers).all()
    # its gradients are those of the block as it stands after training, on a batch of the task
    xs, rs, want = task.batch()
    block.x.copy_(xs)
    block.residual.copy_(rs)
    block.dy.copy_(torch.randn(200, 64, generator=rng(3), device=DEV))
    TrainingStep(torch, [block], torch.device(DEV)).run()
    torch.cuda.synchronize()
    ref = reference(block)
    for name in OUTPUTS:
        assert distance(getattr(block, name), ref[name]) <= FAR, name


def test_tensors_of_another_device_are_refused(monkeypatch):
    """Work is launched on the current device: tensors that live elsewhere are refused before."""
    x, rows = torch.zeros(4, 64, dtype=torch.bfloat16, device=DEV), torch.zeros(4, 2, dtype=torch.int32, device=DEV)
    w, ones = torch.zeros(64, 64, dtype=torch.bfloat16, device=DEV), torch.ones(4, 2, device=DEV)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for call in (lambda: q.nvfp4_route(x, 2), lambda: q.nvfp4_route_backward(x, rows, ones), lambda: q.nvfp4_dispatch(x, rows),
                 lambda: q.nvfp4_combine(x, rows), lambda: q.nvfp4_combine_backward(x, x, rows, ones), lambda: q.nvfp4_rmsnorm(x),
                 lambda: q.nvfp4_rmsnorm_i8(x), lambda: q.nvfp4_rmsnorm_backward(x, x), lambda: q.nvfp4_bf16_linear(x, w),
                 lambda: q.nvfp4_bf16_linear_backward(x, x, q.ACT_SILU)):
        with pytest.raises(ValueError, match="expected cuda:1"):
            call()
