"""GPU tests of what the expert-layer calls do to memory: the training-step
driver's layer of experts allocates nothing in a step, also where its
contractions are split; no step runs over buffers that share memory; an
AdamWGroup does not let go of its tensors' memory."""
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


def group_tensors(torch, dev, bits, n=70_000):
    d = {"params": [torch.ones(n, device=dev)], "grads": [torch.ones(n, device=dev)]}
    if bits == 8:
        for k in ("m", "v"):
            d[k] = [torch.zeros(n, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn)]
            d[k + "_scales"] = [torch.zeros(-(-n // 128), device=dev)]
    else:
        d.update(m=[torch.zeros(n, device=dev)], v=[torch.zeros(n, device=dev)])
    d["copies"] = [torch.zeros(n, dtype=torch.bfloat16, device=dev)]
    return d


OVERLAPS = [
    ("m and v", lambda d, t: d.update(v=d["m"])),
    ("m and v in part", lambda d, t: d.update(m=[t[0:1000]], v=[t[996:1996]])),
    ("params in part", lambda d, t: d.update(params=[t[0:1000]], m=[t[999:1999]])),
    ("params and grads", lambda d, t: d.update(grads=d["params"])),
    ("copies and grads", lambda d, t: d.update(grads=[t[0:1000]], copies=[t[500:1000].view(d["copies"][0].dtype)])),
]


@pytest.mark.parametrize("what", range(len(OVERLAPS)))
def test_refuses_a_step_over_buffers_that_overlap(env, what):
    torch, q, dev = env
    name, change = OVERLAPS[what]
    d = group_tensors(torch, dev, 32, 1000)
    change(d, torch.zeros(4000, device=dev))
    before = {k: v[0].clone() for k, v in d.items()}
    print(f"overlap of {name}", flush=True)
    with pytest.raises(ValueError, match="overlap"):
        q.nvfp4_adamw(q.AdamWGroup(**d), 1, 1e-3)
    torch.cuda.synchronize()
    for k, v in d.items():
        assert torch.equal(v[0], before[k]), k


def test_takes_neighbours_and_shared_gradients(env):
    """Pieces of one buffer that touch, gradients read by two tensors, and
    tensors without elements are no overlap."""
    torch, q, dev = env
    flat, g = torch.zeros(8 * 128, device=dev), torch.ones(128, device=dev)
    cut = [flat[128 * i:128 * (i + 1)] for i in range(6)]
    empty = flat[100:100]
    print("neighbours", flush=True)
    q.nvfp4_adamw(q.AdamWGroup(cut[0:2] + [empty], [g, g, empty], cut[2:4] + [empty], cut[4:6] + [empty]), 1, 1e-3)
    assert not flat[768:].any().item() and flat[:768].all().item()


@pytest.mark.parametrize("bits", [32, 8])
def test_memory_of_a_group_is_not_given_to_others(env, bits):
    """A tensor of a group that is pointed to other memory: the old memory,
    which the next step still writes, stays the group's."""
    torch, q, dev = env
    d = group_tensors(torch, dev, bits)
    group = q.AdamWGroup(**d)
    for kind, (t,) in d.items():
        old, size = t.data_ptr(), t.numel() * t.element_size()
        torch.cuda.synchronize()
        t.data = torch.zeros_like(t)
        others = [torch.empty(size, dtype=torch.uint8, device=dev) for _ in range(8)]
        print(f"group keeps {kind}, bits {bits}", flush=True)
        for o in others:
            assert not (o.data_ptr() < old + size and old < o.data_ptr() + o.numel()), kind
    del group
