"""A block of experts trained and then asked: norm, router, dispatch, two products
with an activation between them and combine, with their gradients, AdamW over
all of its weights, a bias that balances the experts' load, and a few tokens
through the trained block and an int8 head.

The task is synthetic: the block learns a fixed random two-layer map of its input
beside the residual.

    python examples/expert_block.py [--steps 100]
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import quantize_precision_gemm_amd as q  # noqa: E402
from quantize_precision_gemm_amd.step import BF16ExpertBlock, TrainingStep  # noqa: E402


class BlockTask:
    """Inputs x and the outputs that the block should give for them (its residual is x / 2)."""

    def __init__(self, tokens, hidden, seed, device):
        self.g = torch.Generator(device=device)
        self.g.manual_seed(seed)
        self.tokens, self.hidden, self.device = tokens, hidden, device
        self.up = self.randn(2 * hidden, hidden) / hidden ** 0.5
        self.down = 0.5 * self.randn(hidden, 2 * hidden) / hidden ** 0.5

    def randn(self, *shape):
        return torch.randn(shape, generator=self.g, device=self.device)

    def batch(self, tokens=None):
        x = self.randn(tokens or self.tokens, self.hidden).bfloat16()
        want = 1.5 * x.float() + torch.relu(x.float() @ self.up.t()) @ self.down.t()
        return x, (x / 2), want


def build(task, experts, inner, k):
    """The block and its master weights (fp32); its products read bf16 copies that each update writes."""
    h = task.hidden
    master = {"norm_weight": torch.ones(h, device=task.device), "router": 0.05 * task.randn(experts, h),
              "w1": task.randn(experts, inner, h) / h ** 0.5, "b1": torch.zeros(experts, inner, device=task.device),
              "w2": 0.1 * task.randn(experts, h, inner) / inner ** 0.5}
    bf16 = {name: master[name].bfloat16() for name in ("router", "w1", "w2")}
    x, residual, _ = task.batch()
    block = BF16ExpertBlock(q, torch, x, residual, torch.zeros_like(x), master["norm_weight"], bf16["router"], bf16["w1"],
                            master["b1"], bf16["w2"], k, activation=q.ACT_SILU, score=q.SIGMOID,
                            choice_bias=torch.zeros(experts, device=task.device))
    return block, master, bf16


def train(steps=100, tokens=1024, hidden=128, experts=8, inner=256, k=2, lr=2e-3, balance=1e-3, seed=0, device="cuda:0", log=None):
    task = BlockTask(tokens, hidden, seed, device)
    block, master, bf16 = build(task, experts, inner, k)
    grads = [block.dnorm, block.drouter[0], block.dw1, block.db1, block.dw2]
    group = q.AdamWGroup.with_states(list(master.values()), grads,
                                     copies=[bf16.get(name) for name in master])
    step_of = TrainingStep(torch, [block], device)
    losses = []
    for step in range(1, steps + 1):
        x, residual, want = task.batch()
        block.x.copy_(x)
        block.residual.copy_(residual)
        for _, op in block.forward_ops():
            op()
        error = block.y.float() - want
        losses.append(error.square().mean())
        block.dy.copy_(error * (2.0 / error.numel() * 1024))  # (scaled into bf16's range; AdamW does not mind)
        step_of.run()
        q.nvfp4_adamw(group, step, lr, weight_decay=0.0)
        # experts with more than their share become less likely
        load = torch.diff(block.routing.ends, prepend=block.routing.ends.new_zeros(1)).float()
        block.choice_args["bias"].sub_(balance * torch.sign(load - load.mean()))
        if log and (step == 1 or step % 20 == 0):
            log(f"step {step}: loss {losses[-1].item():.5f}, largest load {(load.max() / load.mean()).item():.2f} of the mean")
    return [v.item() for v in losses], block, task


def ask(block, x, residual, head):
    """A few tokens through the trained block, normalised into int8, and an int8 head: what a decoding step does."""
    n, h = q.nvfp4_rmsnorm(x, block.norm_weight, block.eps, residual=residual)
    logits = q.nvfp4_bf16_linear(n, block.router, out_dtype=torch.float32)
    r = q.nvfp4_route(logits, block.k, **block.route_args, **block.choice_args)
    a = q.nvfp4_bf16_linear(q.nvfp4_dispatch(n, r.rows), block.w1, ends=r.ends, bias=block.b1, activation=block.activation)
    y = q.nvfp4_combine(q.nvfp4_bf16_linear(a, block.w2, ends=r.ends), r.rows, r.weights, residual=h)
    n8, _ = q.nvfp4_rmsnorm_i8(y, block.norm_weight, block.eps)
    return y, q.nvfp4_i8_gemm(n8, head, torch.float32)


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--steps", type=int, default=100)
    a = p.parse_args()
    losses, block, task = train(a.steps, log=print)
    x, residual, want = task.batch(3)
    y, answers = ask(block, x, residual, q.nvfp4_i8_quantize(task.randn(64, task.hidden).bfloat16()))
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f}; three tokens: off by {(y.float() - want).square().mean().item():.4f}, "
          f"answers {tuple(answers.shape)}")


if __name__ == "__main__":
    main()
