"""GPU tests of AdamW steps whose gradients, moments or eps leave fp32's range
or 8-bit states' (nvfp4_adamw): what the other elements of a block keep, and
what the element itself is held as.

No tolerances: runs that must agree execute the same fp32 operations, and are
compared bit for bit.
"""
import pytest

from tests.gpu_util import ensure_built

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")
HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
TOP = 0.03125  # the largest value of the block, steady from step to step


@pytest.fixture(scope="module")
def env():
    import torch
    ensure_built()
    import quantize_precision_gemm_amd as q
    return torch, q, torch.device("cuda:0")


def bits_of(torch, t):
    return t.view(torch.uint8)


class Run:
    """Tensors of n elements whose states have seen some steps.  In each block
    one element has the gradient TOP at every step (its moments are TOP: the
    block's scales stay); the others' are below half of it, element `at` has
    none."""

    def __init__(self, torch, q, dev, bits, count, n, at):
        g = torch.Generator(device=dev)
        g.manual_seed(3)
        self.torch, self.q, self.at, self.gen = torch, q, at, g
        self.params = [torch.randn(n, generator=g, device=dev) for _ in range(count)]
        self.grads = [torch.zeros(n, device=dev) for _ in range(count)]
        self.group = q.AdamWGroup.with_states(self.params, self.grads, bits=bits)
        self.number = 0
        for _ in range(3):
            self.step()

    def step(self, value=None):
        torch = self.torch
        for grad in self.grads:
            grad.copy_(0.004 * torch.randn(grad.shape, generator=self.gen, device=grad.device).clamp(-3, 3))
            grad[::128] = TOP
            grad[self.at] = 0.0 if value is None else value
        self.number += 1
        self.q.nvfp4_adamw(self.group, self.number, **HYPER)

    def state(self):
        g = self.group
        lists = [self.params, g.m, g.v] + ([g.m_scales, g.v_scales] if g.bits == 8 else [])
        return [[t.clone() for t in x] for x in lists]


@pytest.mark.parametrize("value", [NAN, INF, -INF, 5e19, -1e20, 3.4e38])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("count", [1, 60])  # 60: from the table in device memory
def test_one_gradient_out_of_range_leaves_the_others_alone(env, value, bits, count):
    """For the steps after it too: parameters, moments and scales of every
    other element have the bits of a run in which that gradient was 0.  One
    that is not finite makes its own parameter NaN; one whose square alone
    leaves fp32's range does not."""
    torch, q, dev = env
    n, at = 1000, 301
    clean, run = (Run(torch, q, dev, bits, count, n, at) for _ in range(2))
    other = torch.arange(n, device=dev) != at
    for k, g in enumerate([value] + [None] * 5):
        print(f"adamw gradient {value}, bits {bits}, count {count}, step {k}", flush=True)
        run.step(g)
        clean.step()
        for i, (a, b) in enumerate(zip(run.state(), clean.state())):
            for x, y in zip(a, b):
                if x.numel() == n:
                    x, y = x[other], y[other]
                assert torch.equal(bits_of(torch, x), bits_of(torch, y)), f"list {i}, step {k}"
        for p in run.params:
            assert torch.isfinite(p[at]).item() == (value == value and abs(value) != INF), f"step {k}"


@pytest.mark.parametrize("n", [1, 128, 500])
@pytest.mark.parametrize("value", [1e20, -3e38])
def test_blocks_of_overflowing_squares_stay_finite_and_recover(env, n, value):
    """Every gradient's square overflows: 8-bit states hold no NaN, the
    parameters only decay at that step, and later steps train again."""
    torch, q, dev = env
    p, g = torch.ones(n, device=dev), torch.full((n,), value, device=dev)
    group = q.AdamWGroup.with_states([p], [g], bits=8)
    print(f"adamw all {value} n {n}", flush=True)
    q.nvfp4_adamw(group, 1, **HYPER)
    keep = torch.tensor(1 - HYPER["lr"] * HYPER["weight_decay"], dtype=torch.float32, device=dev)
    assert torch.equal(p, torch.ones(n, device=dev) * keep)
    for t in (group.m[0], group.v[0]):
        assert torch.isfinite(t.float()).all().item()
    g.fill_(0.5)
    before = p.clone()
    for step in (2, 3, 4):
        q.nvfp4_adamw(group, step, **HYPER)
    assert torch.isfinite(p).all().item() and (p < before).all().item()


@pytest.mark.parametrize("bits", [32, 8])
def test_roots_up_to_the_largest_square(env, bits):
    """Gradients of 1.8e19, whose squares fp32 just holds, until the root has
    grown to them: its square stays finite in 8 bits as in 32."""
    torch, q, dev = env
    p, g = torch.ones(256, device=dev), torch.full((256,), 1.8e19, device=dev)
    group = q.AdamWGroup.with_states([p], [g], bits=bits)
    for step in range(1, 121):
        print(f"adamw large root, bits {bits}, step {step}", flush=True)
        before = p.clone()
        q.nvfp4_adamw(group, step, **HYPER)
        assert torch.isfinite(p).all().item() and (p < before).all().item()
        # m / root, corrected, is 1; 8-bit moments are off by 2^-4 each at most and
        # the root may be held as 7/8 of itself, so twice the rate bounds a step
        assert ((before - p) <= 2 * HYPER["lr"] + HYPER["lr"] * HYPER["weight_decay"]).all().item()
    assert torch.isfinite(group.v[0].float()).all().item()


def test_states_out_of_range_from_elsewhere(env):
    """Roots whose squares overflow and first moments next to fp32's largest,
    as scales that were not written here may give them, come back into range."""
    torch, q, dev = env
    p, g = torch.ones(256, device=dev), torch.full((256,), 0.01, device=dev)

    def codes(value):
        return torch.full((256,), value, device=dev).to(torch.float8_e4m3fn)
    m, v = codes(448.0), codes(448.0)
    ms = torch.tensor([2.0 ** 119, 1.0], device=dev)  # 448 of them: 1.75 * 2^127
    vs = torch.tensor([2.0 ** 50, 2.0 ** 100], device=dev)
    group = q.AdamWGroup([p], [g], [m], [v], [ms], [vs])
    for step in range(1, 5):
        print(f"adamw foreign states step {step}", flush=True)
        q.nvfp4_adamw(group, step, lr=0.0, weight_decay=0.0, beta1=0.9, beta2=0.95)
        assert torch.isfinite(m.float()).all().item() and torch.isfinite(v.float()).all().item()
        assert torch.isfinite(ms).all().item() and (vs <= 2.0 ** 55).all().item()
    assert torch.equal(p, torch.ones(256, device=dev))


@pytest.mark.parametrize("bits", [32, 8])
def test_an_eps_below_fp32_is_not_zero(env, bits):
    """A parameter that never had a gradient is not divided 0 by 0."""
    torch, q, dev = env
    p, g = torch.ones(200, device=dev), torch.zeros(200, device=dev)
    g[::2] = 0.5
    group = q.AdamWGroup.with_states([p], [g], bits=bits)
    print(f"adamw eps 1e-60 bits {bits}", flush=True)
    for step in (1, 2):
        q.nvfp4_adamw(group, step, lr=1e-3, eps=1e-60, weight_decay=0.0)
    assert torch.equal(p[1::2], torch.ones(100, device=dev))
    assert (p[::2] < 1).all().item() and torch.isfinite(p).all().item()
