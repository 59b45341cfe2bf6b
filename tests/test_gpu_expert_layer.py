"""The expert layer of examples/expert_layer.py: its three passes through
the training-step driver, its training and its answers in int8."""
import os
import sys

import pytest

from tests.gpu_util import ROOT, ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    ensure_built()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import expert_layer
    import quantize_precision_gemm_amd as q
    return torch, q, expert_layer


def test_experts_in_a_training_step(env):
    """BF16Experts beside a plain bf16 layer in one TrainingStep: the outputs
    of the calls made one by one."""
    torch, q, _ = env
    from quantize_precision_gemm_amd.step import BF16Experts, BF16Linear, TrainingStep
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev)
    g.manual_seed(3)

    def rnd(*s):
        return torch.randn(s, generator=g, device=dev).bfloat16()
    T, K, N, E = 300, 256, 136, 3
    ends = torch.tensor([120, 120, 300], dtype=torch.int32, device=dev)
    experts = BF16Experts(q, torch, rnd(T, K), rnd(E, N, K), rnd(T, N), ends)
    dense = BF16Linear(q, torch, rnd(T + 4, K), rnd(N, K), rnd(T + 4, N))  # (its tokens come in eights)
    for serial in (False, True):
        for t in (experts.y, experts.dx, experts.dw):
            t.zero_()
        print(f"experts in a step, serial {serial}", flush=True)
        TrainingStep(torch, [dense, experts], dev, serial_gemms=serial).run()
        torch.cuda.synchronize()
        assert torch.equal(experts.y, q.nvfp4_bf16_grouped_gemm(q.FPROP, experts.x, experts.w, ends))
        assert torch.equal(experts.dx, q.nvfp4_bf16_grouped_gemm(q.DGRAD, experts.dy, experts.w, ends))
        assert torch.equal(experts.dw, q.nvfp4_bf16_grouped_gemm(q.WGRAD, experts.dy, experts.x, ends, torch.float32))


@pytest.mark.parametrize("bits", [32, 8])
def test_training_learns_the_maps(env, bits):
    """From zero weights the loss starts at the targets' variance (1) and has
    to fall to a twentieth of it; the int8 answers stay near the bf16 ones:
    codes of 127 steps put an error of about 1 / (127 sqrt(12) / 3) = 0.7 % of a
    typical value on each factor, 2 % leaves twice both."""
    torch, q, ex = env
    print(f"expert layer training, {bits}-bit states", flush=True)
    losses, master, task = ex.train(steps=60, bits=bits)
    assert 0.8 < losses[0] < 1.25
    assert losses[-1] < 0.05, losses[::10]
    x, ends, _ = task.batch()
    bf16 = q.nvfp4_bf16_grouped_gemm(q.FPROP, x, master.bfloat16(), ends, torch.float32)
    int8 = ex.answer_in_int8(master, x, ends)
    assert ((int8 - bf16).norm() / bf16.norm()).item() < 0.02


@pytest.mark.parametrize("what", ["grouped", "split", "quantize", "int8"])
def test_outputs_made_for_another_stream_are_its_own(env, what):
    """Memory freed on the current stream, where work on it is still waiting,
    is not given to a call on another stream."""
    torch, q, _ = env
    dev = torch.device("cuda:0")
    T, E, N, K = (4096, 1, 256, 128) if what == "split" else (512, 2, 256, 128)
    x = torch.randn(T, K, device=dev).bfloat16()
    dy = torch.randn(T, N, device=dev).bfloat16()
    ends = torch.tensor([T] * E, dtype=torch.int32, device=dev)
    xq, wq = q.nvfp4_i8_quantize(x), q.nvfp4_i8_quantize(dy[:N, :K].contiguous())
    if what == "split":
        assert q.nvfp4_bf16_grouped_gemm_workspace(q.WGRAD, E, T, N, K) > 0

    def call(stream):
        if what in ("grouped", "split"):
            return [q.nvfp4_bf16_grouped_gemm(q.WGRAD, dy, x, ends, torch.float32, stream=stream)]
        if what == "quantize":
            t = q.nvfp4_i8_quantize(x, stream=stream)
            return [t.codes, t.scales]
        return [q.nvfp4_i8_gemm(xq, wq, torch.float32, stream=stream)]
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    sizes = [t.numel() * t.element_size() for t in want]
    if what == "split":
        sizes.append(q.nvfp4_bf16_grouped_gemm_workspace(q.WGRAD, E, T, N, K))
    print(f"another stream: {what} {sizes}", flush=True)
    held = [torch.empty(n, dtype=torch.uint8, device=dev) for n in sizes]
    torch.cuda._sleep(20_000_000)  # about 10 ms
    for t in held:
        t.fill_(255)
    del held, t
    got = call(side)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_inputs_dropped_before_another_stream_has_read_them(env):
    """Inputs that are freed and overwritten on the current stream while the
    work that reads them waits on another one."""
    torch, q, _ = env
    dev = torch.device("cuda:0")
    T, E, N, K = 512, 2, 256, 128
    x, dy = torch.randn(T, K, device=dev).bfloat16(), torch.randn(T, N, device=dev).bfloat16()
    ends = torch.tensor([100, T], dtype=torch.int32, device=dev)
    w = q.nvfp4_i8_quantize(dy[:N, :K].contiguous())
    want = [q.nvfp4_bf16_grouped_gemm(q.WGRAD, dy, x, ends), q.nvfp4_i8_gemm(q.nvfp4_i8_quantize(x), w)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for which in range(2):
        print(f"inputs dropped {which}", flush=True)
        torch.cuda.empty_cache()
        copies = [t.clone() for t in (x, dy, ends)]
        sizes = [t.numel() * t.element_size() for t in copies]
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)  # about 10 ms
        if which == 0:
            got = q.nvfp4_bf16_grouped_gemm(q.WGRAD, copies[1], copies[0], copies[2], stream=side)
        else:
            got = q.nvfp4_i8_gemm(q.nvfp4_i8_quantize(copies[0], stream=side), w, stream=side)
        del copies
        over = [torch.zeros(n, dtype=torch.uint8, device=dev) for n in sizes]
        torch.cuda.synchronize()
        assert torch.equal(got, want[which])
        del over
