"""An expert layer trained and then served: the ragged products of its three
passes in bf16, AdamW over fp32 master weights with states in 8 or 32 bits,
and the trained weights answering in 8-bit integers.

The task is synthetic: every token is routed to one expert by a fixed random
projection, and each expert has to learn a linear map of its own.  Tokens are
drawn anew for each step, so the experts' shares change from step to step.

    python examples/expert_layer.py [--steps 60] [--bits 8]
"""
import argparse
import math
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import quantize_precision_gemm_amd as q  # noqa: E402
from quantize_precision_gemm_amd.step import BF16Experts  # noqa: E402


class ExpertTask:
    """Tokens (sorted by the expert they go to) and the outputs they should get."""

    def __init__(self, tokens, experts, outputs, inputs, seed, device):
        self.g = torch.Generator(device=device)
        self.g.manual_seed(seed)
        self.tokens, self.inputs, self.device = tokens, inputs, device
        self.router = self._randn(inputs, experts)
        self.maps = (self._randn(experts, outputs, inputs) / inputs ** 0.5).bfloat16()

    def _randn(self, *shape):
        return torch.randn(shape, generator=self.g, device=self.device)

    def batch(self):
        x = self._randn(self.tokens, self.inputs).bfloat16()
        expert = (x.float() @ self.router).argmax(1)
        order = torch.argsort(expert, stable=True)
        ends = torch.cumsum(torch.bincount(expert, minlength=self.router.shape[1]), 0).int()
        x = x[order].contiguous()
        return x, ends, q.nvfp4_bf16_grouped_gemm(q.FPROP, x, self.maps, ends, torch.float32)


def clip_factor(grads, limit):
    """limit / norm where the norm is above it (a device scalar: no step waits
    for the host); NaN where the norm is not finite, which leaves the step out."""
    norm = torch.linalg.vector_norm(torch.stack([torch.linalg.vector_norm(g) for g in grads]))
    return torch.where(torch.isfinite(norm), limit / norm.clamp(min=limit), math.nan).reshape(1)


def train(steps=60, bits=8, tokens=4096, experts=6, outputs=512, inputs=256, lr=5e-3, seed=0, device="cuda:0", log=None):
    """Returns (the loss of each step, the master weights E x N x K, the task)."""
    task = ExpertTask(tokens, experts, outputs, inputs, seed, device)
    master = torch.zeros(experts, outputs, inputs, device=device)
    weight = master.bfloat16()  # what the products read: a copy that each update writes
    layer = BF16Experts(q, torch, torch.empty(tokens, inputs, dtype=torch.bfloat16, device=device), weight,
                        torch.empty(tokens, outputs, dtype=torch.bfloat16, device=device),
                        torch.empty(experts, dtype=torch.int32, device=device))
    group = q.AdamWGroup.with_states([master], [layer.dw], bits=bits, copies=[weight])
    losses = []
    for step in range(1, steps + 1):
        x, ends, want = task.batch()
        layer.x.copy_(x)
        layer.ends.copy_(ends)
        for _, op in layer.forward_ops():
            op()
        error = layer.y.float() - want
        losses.append(error.square().mean())
        layer.dy.copy_(error * (2.0 / tokens))
        for _, op in layer.dgrad_ops() + layer.wgrad_ops():  # (dgrad: what a layer before this one would get)
            op()
        q.nvfp4_adamw(group, step, lr, weight_decay=0.0, grad_scale=clip_factor([layer.dw], 10.0))
        if log and (step == 1 or step % 10 == 0):
            log(f"step {step}: loss {losses[-1].item():.5f}")
    return [v.item() for v in losses], master, task


def answer_in_int8(master, x, ends):
    """The layer's outputs with weights and tokens as int8, expert by expert."""
    weights = [q.nvfp4_i8_quantize(w.bfloat16()) for w in master]
    out, begin = [], 0
    for w, end in zip(weights, ends.tolist()):
        out.append(q.nvfp4_i8_gemm(q.nvfp4_i8_quantize(x[begin:end]), w, torch.float32))
        begin = end
    return torch.cat(out)


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--steps", type=int, default=60)
    p.add_argument("--bits", type=int, choices=(8, 32), default=8, help="bits of the AdamW states")
    a = p.parse_args()
    losses, master, task = train(a.steps, a.bits, log=print)
    x, ends, want = task.batch()
    got = answer_in_int8(master, x, ends)
    bf16 = q.nvfp4_bf16_grouped_gemm(q.FPROP, x, master.bfloat16(), ends, torch.float32)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f}; int8 answers differ from the bf16 ones by "
          f"{((got - bf16).norm() / bf16.norm()).item():.4f} (relative norm)")


if __name__ == "__main__":
    main()
