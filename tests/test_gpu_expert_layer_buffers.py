"""GPU tests of what the expert-layer calls do to memory: the training-step
driver's layer of experts allocates nothing in a step, also where its
contractions are split."""
import pytest

from tests.gpu_util import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    ensure_built()
    import quantize_precision_gemm_amd as q
    return torch, q, torch.device("cuda:0")


@pytest.mark.parametrize("serial", [False, True])
def test_a_step_of_experts_allocates_nothing(env, serial):
    """dgrad and wgrad both split, side by side on two streams: the outputs of
    the calls made one by one, and no block is taken from the allocator."""
    torch, q, dev = env
    from quantize_precision_gemm_amd.step import BF16Experts, TrainingStep
    g = torch.Generator(device=dev)
    g.manual_seed(3)

    def rnd(*s):
        return torch.randn(s, generator=g, device=dev).bfloat16()
    T, K, N, E = 8192, 128, 4104, 2
    ends = torch.tensor([900, T], dtype=torch.int32, device=dev)
    layer = BF16Experts(q, torch, rnd(T, K), rnd(E, N, K), rnd(T, N), ends)
    few = BF16Experts(q, torch, rnd(T, 136), rnd(E, 72, 136), rnd(T, 72), ends)
    assert q.nvfp4_bf16_grouped_gemm_workspace(q.DGRAD, E, T, N, K) > 0
    assert q.nvfp4_bf16_grouped_gemm_workspace(q.WGRAD, E, T, 72, 136) > 0
    step = TrainingStep(torch, [layer, few], dev, serial_gemms=serial)
    step.run()
    torch.cuda.synchronize()
    before = torch.cuda.memory_stats()["allocation.all.allocated"]
    for i in range(3):
        for x in (layer, few):
            for t in (x.y, x.dx, x.dw):
                t.fill_(-7.0)
        print(f"step of experts {i}, serial {serial}", flush=True)
        step.run()
    torch.cuda.synchronize()
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == before
    for x in (layer, few):
        assert torch.equal(x.y, q.nvfp4_bf16_grouped_gemm(q.FPROP, x.x, x.w, ends))
        assert torch.equal(x.dx, q.nvfp4_bf16_grouped_gemm(q.DGRAD, x.dy, x.w, ends))
        assert torch.equal(x.dw, q.nvfp4_bf16_grouped_gemm(q.WGRAD, x.dy, x.x, ends, torch.float32))
