"""GPU tests of the AdamW step (nvfp4_adamw) against the formulas in 64 bits,
and against the same fp32 operations one by one, which it must equal.

Tolerances, with h = 2^-24 (half a step of fp32) and every factor of the step
rounded once (h more each):
- m: two products and a sum, each a rounding and a rounded factor:
  <= 4 h (|beta1 m| + |(1 - beta1) g|); g itself is off by h after the scale.
- v: the same with the square (2 h of g, 1 of the square): <= 7 h v.
- p: the quotient's relative error is at most that of m (relative to the sum
  of its magnitudes) plus half of v's, the root, the factor, the product, the
  sum with eps, the quotient, the rate and its product: <= 12 h; the two terms
  of p and their difference 4 h of their size.
- bf16 results: 2^-8 of the value more.
- 8-bit states: half a step of E4M3, 2^-4 of the value or 2^-10 of the scale;
  a nonzero root below 2^-9 of the scale is held as that: within 2^-9 of it.
"""
import math

import numpy as np
import pytest

from tests.gpu_util import ensure_built

pytestmark = pytest.mark.gpu

H = 2.0 ** -24
HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)


@pytest.fixture(scope="module")
def env():
    import torch
    ensure_built()
    import quantize_precision_gemm_amd as q
    return torch, q, torch.device("cuda:0")


def blocks(torch, x):
    """x (flat) as rows of 128, the last one filled with zeros."""
    n = x.numel()
    full = torch.zeros(-(-n // 128) * 128, dtype=x.dtype, device=x.device)
    full[:n] = x
    return full.view(-1, 128)


def values(torch, codes, scales):
    """What 8-bit codes and scales stand for."""
    return (blocks(torch, codes.float().double()) * scales.double()[:, None]).flatten()[: codes.numel()]


def tensors(torch, dev, sizes, p_dtype, g_dtype, bits, copy, seed, offset=0):
    """Lists of tensors, `offset` elements into their buffers (to miss the wide alignment)."""
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def place(x, dtype):
        buf = torch.zeros(x.numel() + offset, device=dev, dtype=dtype)
        buf[offset:] = x.to(dtype)
        return buf[offset:]

    def place8(x):
        buf = torch.zeros(x.numel() + offset, device=dev, dtype=torch.uint8)
        buf[offset:] = x.to(torch.float8_e4m3fn).view(torch.uint8)
        return buf[offset:].view(torch.float8_e4m3fn)
    d = {k: [] for k in ("params", "grads", "m", "v", "m_scales", "v_scales", "copies")}
    for n in sizes:
        p, gr = torch.randn(n, generator=g, device=dev), 0.01 * torch.randn(n, generator=g, device=dev)
        m, r = 0.002 * torch.randn(n, generator=g, device=dev), (0.01 * torch.randn(n, generator=g, device=dev)).abs()
        gr *= torch.exp(2 * torch.randn(n, generator=g, device=dev))  # gradients of many sizes
        d["params"].append(place(p, p_dtype))
        d["grads"].append(place(gr, g_dtype))
        if bits == 8:
            sm = torch.full((-(-n // 128),), 2.0 ** -14, device=dev)
            d["m"].append(place8(m * 2.0 ** 14))
            d["v"].append(place8(r * 2.0 ** 13))
            d["m_scales"].append(sm)
            d["v_scales"].append(sm * 2)
        else:
            d["m"].append(place(m, torch.float32))
            d["v"].append(place(r * r, torch.float32))
        d["copies"].append(place(p * 0, torch.bfloat16) if copy else None)
    if bits == 32:
        d["m_scales"] = d["v_scales"] = None
    return d


def clone(d):
    return {k: None if v is None else [None if t is None else t.clone() for t in v] for k, v in d.items()}


def scales_of(torch, x):
    """The smallest power of two 2^j >= 2^-126 with max |x| <= 448 * 2^j per block."""
    top = blocks(torch, x).abs().amax(1)
    return torch.exp2(torch.ceil(torch.log2(top / 448.0)).clamp(min=-126.0))


def check_tensor(torch, old, new, i, step, gs, bits, hyper):
    b1, b2 = hyper["beta1"], hyper["beta2"]
    p0, g = old["params"][i].double(), old["grads"][i].double() * gs
    if bits == 8:
        m0 = values(torch, old["m"][i], old["m_scales"][i])
        v0 = values(torch, old["v"][i], old["v_scales"][i]) ** 2
    else:
        m0, v0 = old["m"][i].double(), old["v"][i].double()
    m, v = b1 * m0 + (1 - b1) * g, b2 * v0 + (1 - b2) * g * g
    m_size = b1 * m0.abs() + (1 - b1) * g.abs()
    tiny = 2.0 ** -148  # results below fp32's normal range
    rate, root = hyper["lr"] / (1 - b1 ** step), v.sqrt() / math.sqrt(1 - b2 ** step)
    den = root + hyper["eps"]
    p = p0 * (1 - hyper["lr"] * hyper["weight_decay"]) - rate * m / den
    p_tol = 4 * H * (p0.abs() + rate * m.abs() / den) + 17 * H * rate * m_size / den + tiny
    if new["params"][i].dtype == torch.bfloat16:
        p_tol = p_tol + 2.0 ** -8 * (p.abs() + p_tol)
    assert ((new["params"][i].double() - p).abs() <= p_tol).all().item(), f"p of tensor {i}"
    if new["copies"][i] is not None:
        assert torch.equal(new["copies"][i], new["params"][i].bfloat16()), f"copy of tensor {i}"
    m_tol, v_tol = 5 * H * m_size + tiny, 7 * H * v + tiny
    if bits == 32:
        assert ((new["m"][i].double() - m).abs() <= m_tol).all().item(), f"m of tensor {i}"
        assert ((new["v"][i].double() - v).abs() <= v_tol).all().item(), f"v of tensor {i}"
        return
    r = v.sqrt()
    r_tol = 5 * H * r + tiny
    for name, x, tol in (("m", m, m_tol), ("v", r, r_tol)):
        s = scales_of(torch, x)
        got_s = new[name + "_scales"][i].double()
        same = got_s == s
        # a block whose maximum lies within its rounding of a border may take either scale
        near = (blocks(torch, x).abs().amax(1) / (448 * s) > 1 - 2.0 ** -20) | \
               (blocks(torch, x).abs().amax(1) / (224 * s) < 1 + 2.0 ** -20)
        assert (same | near).all().item(), f"{name} scales of tensor {i}"
        val = values(torch, new[name][i], new[name + "_scales"][i])
        step_size = got_s.repeat_interleave(128)[: x.numel()]
        least = 2.0 ** -10 if name == "m" else 2.0 ** -9
        assert ((val - x).abs() <= torch.maximum(2.0 ** -4 * x.abs(), least * step_size) + 2 * tol).all().item(), \
            f"{name} of tensor {i}"
        if name == "v":
            assert ((val > 0) | (x == 0)).all().item(), "a nonzero root is held as zero"


SIZES = [1, 3, 127, 128, 129, 1023, 1024, 1025, 5000, 0, 2, 40000]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("p_dtype,g_dtype,copy", [("float32", "float32", True), ("float32", "bfloat16", False),
                                                  ("bfloat16", "bfloat16", False), ("bfloat16", "float32", False)])
@pytest.mark.parametrize("offset", [0, 1])
def test_step(env, bits, p_dtype, g_dtype, copy, offset):
    torch, q, dev = env
    d = tensors(torch, dev, SIZES, getattr(torch, p_dtype), getattr(torch, g_dtype), bits, copy, 7, offset)
    old = clone(d)
    gs = torch.tensor([0.37], device=dev)
    print(f"adamw {bits} {p_dtype} {g_dtype} offset {offset}", flush=True)
    q.nvfp4_adamw(q.AdamWGroup(**d), 12, grad_scale=gs, **HYPER)
    torch.cuda.synchronize()
    for i in range(len(SIZES)):
        check_tensor(torch, old, d, i, 12, float(gs.item()), bits, HYPER)
        assert torch.equal(old["grads"][i], d["grads"][i])


@pytest.mark.parametrize("bits", [32, 8])
def test_equals_the_same_operations_one_by_one(env, bits):
    """fp32 on the CPU, each operation rounded once: the kernel's bits."""
    torch, q, dev = env
    n, step = 30000, 5
    d = tensors(torch, dev, [n], torch.float32, torch.float32, bits, False, 3)
    f = np.float32
    host = {k: v[0].float().cpu().numpy() for k, v in d.items() if v is not None and v[0] is not None}
    print(f"adamw bits {bits}", flush=True)
    q.nvfp4_adamw(q.AdamWGroup(**d), step, **HYPER)
    b1, b2 = HYPER["beta1"], HYPER["beta2"]
    g, m, v = host["grads"], host["m"], host["v"]
    if bits == 8:
        m = m * np.repeat(host["m_scales"], 128)[:n]
        v = v * np.repeat(host["v_scales"], 128)[:n]
        v = v * v
    m = f(b1) * m + f(1 - b1) * g
    v = f(b2) * v + f(1 - b2) * (g * g)
    r = np.sqrt(v)
    p = host["params"] * f(1 - HYPER["lr"] * HYPER["weight_decay"]) - f(HYPER["lr"] / (1 - b1 ** step)) * (
        m / (r * f(1 / math.sqrt(1 - b2 ** step)) + f(HYPER["eps"])))
    np.testing.assert_array_equal(d["params"][0].cpu().numpy(), p)
    if bits == 32:
        np.testing.assert_array_equal(d["m"][0].cpu().numpy(), m)
        np.testing.assert_array_equal(d["v"][0].cpu().numpy(), v)
        return
    for name, x in (("m", m), ("v", r)):
        x = torch.from_numpy(x)
        s = scales_of(torch, x.double()).float()
        np.testing.assert_array_equal(d[name + "_scales"][0].cpu().numpy(), s.numpy())
        y = x / s.repeat_interleave(128)[:n]
        if name == "v":
            y = torch.where(y > 0, y.clamp(min=2.0 ** -9), y)
        want = y.to(torch.float8_e4m3fn).view(torch.uint8)
        np.testing.assert_array_equal(d[name][0].cpu().view(torch.uint8).numpy(), want.numpy())


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors_equal_one_by_one(env, bits):
    """More tensors than one launch takes; each as if it were alone."""
    torch, q, dev = env
    sizes = [(37 * i) % 3001 for i in range(131)]
    d = tensors(torch, dev, sizes, torch.float32, torch.float32, bits, True, 5)
    one = clone(d)
    print(f"adamw 131 tensors bits {bits}", flush=True)
    q.nvfp4_adamw(q.AdamWGroup(**d), 3, **HYPER)
    for i in range(len(sizes)):
        q.nvfp4_adamw(q.AdamWGroup(**{k: None if v is None else v[i:i + 1] for k, v in one.items()}), 3, **HYPER)
    torch.cuda.synchronize()
    for k, v in d.items():
        if v is not None:
            for i, t in enumerate(v):
                a, b = (x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x for x in (t, one[k][i]))
                assert torch.equal(a, b), f"{k} of tensor {i}"


@pytest.mark.parametrize("bits", [32, 8])
def test_first_steps_from_zero_states(env, bits):
    """Ten steps from new states against the 64-bit optimizer: in 32 bits to
    rounding; in 8 bits every step is checked from the state it started with."""
    torch, q, dev = env
    n = 1000
    g = torch.Generator(device=dev)
    g.manual_seed(2)
    p, grad = torch.randn(n, generator=g, device=dev), torch.empty(n, device=dev)
    grp = q.AdamWGroup.with_states([p], [grad], bits=bits)
    d = {"params": grp.params, "grads": grp.grads, "m": grp.m, "v": grp.v, "copies": grp.copies,
         "m_scales": grp.m_scales if bits == 8 else None, "v_scales": grp.v_scales if bits == 8 else None}
    for step in range(1, 11):
        grad.copy_(torch.randn(n, generator=g, device=dev))
        grad[::7] = 0.0
        old = clone(d)
        print(f"adamw step {step} bits {bits}", flush=True)
        q.nvfp4_adamw(grp, step, **HYPER)
        check_tensor(torch, old, d, 0, step, 1.0, bits, HYPER)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_a_scale_that_is_not_finite_leaves_the_step_out(env, bits, value):
    torch, q, dev = env
    d = tensors(torch, dev, [500, 3], torch.float32, torch.float32, bits, True, 1)
    old = clone(d)
    print(f"adamw scale {value}", flush=True)
    q.nvfp4_adamw(q.AdamWGroup(**d), 1, grad_scale=torch.tensor([value], device=dev), **HYPER)
    torch.cuda.synchronize()
    for k, v in d.items():
        if v is not None:
            for a, b in zip(v, old[k]):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), k


@pytest.mark.parametrize("bits", [32, 8])
def test_a_gradient_that_is_not_finite_stays_with_its_element(env, bits):
    torch, q, dev = env
    n, at = 1000, 300
    d = tensors(torch, dev, [n], torch.float32, torch.float32, bits, False, 1)
    clean = clone(d)
    d["grads"][0][at] = float("nan")
    print(f"adamw NaN gradient bits {bits}", flush=True)
    q.nvfp4_adamw(q.AdamWGroup(**d), 1, **HYPER)
    q.nvfp4_adamw(q.AdamWGroup(**clean), 1, **HYPER)
    other = torch.arange(n, device=dev) != at
    assert torch.equal(d["params"][0][other], clean["params"][0][other])
    assert torch.isnan(d["params"][0][at]).item()
    if bits == 32:
        assert torch.equal(d["m"][0][other], clean["m"][0][other])
        assert torch.isnan(d["m"][0][at]).item() and torch.isnan(d["v"][0][at]).item()
    else:  # its block's other values share the largest scale
        far = torch.arange(n, device=dev) // 128 != at // 128
        for k in ("m", "v"):
            assert torch.equal(d[k][0].float()[far], clean[k][0].float()[far])
            assert torch.isnan(d[k][0].float()[at]).item()
            assert torch.isfinite(d[k + "_scales"][0]).all().item()
            assert torch.isfinite(d[k][0].float()[other]).all().item()


def test_zero_gradients_on_zero_states_only_decay(env):
    torch, q, dev = env
    p = torch.randn(777, device=dev)
    old = p.clone()
    for bits in (32, 8):
        grp = q.AdamWGroup.with_states([p], [torch.zeros(777, device=dev)], bits=bits)
        print(f"adamw zeros bits {bits}", flush=True)
        q.nvfp4_adamw(grp, 1, **HYPER)
        old = old * torch.tensor(np.float32(1 - HYPER["lr"] * HYPER["weight_decay"]), device=dev)
        assert torch.equal(p, old)
        assert not grp.m[0].float().any().item() and not grp.v[0].float().any().item()


def test_extreme_gradients(env):
    """Gradients whose squares leave fp32's range on either side, and blocks
    that mix them: 8-bit states stay finite where the 32-bit ones do, a root
    beside a large one is not lost, subnormal blocks are held."""
    torch, q, dev = env
    g = torch.zeros(512, device=dev)
    g[:128] = 1e-30                     # squares underflow
    g[128:256] = 1e-3
    g[128] = 3e4                        # one large value in a block of small ones
    g[256:384] = 2.0 ** -130            # subnormal gradients
    g[384:512:2] = 1e18
    for bits in (32, 8):
        p = torch.ones(512, device=dev)
        grp = q.AdamWGroup.with_states([p], [g], bits=bits)
        print(f"adamw extremes bits {bits}", flush=True)
        for step in (1, 2):
            q.nvfp4_adamw(grp, step, **HYPER)
        assert torch.isfinite(p).all().item()
        # |m| / (sqrt(v) + eps), corrected, stays near 1; twice the rate bounds each step
        assert ((p - 1).abs() <= 2 * (2 * HYPER["lr"] + HYPER["lr"] * HYPER["weight_decay"])).all().item()
        assert torch.isfinite(grp.v[0].float()).all().item()


@pytest.mark.parametrize("p_dtype,g_dtype", [("float32", "bfloat16"), ("bfloat16", "float32"),
                                             ("bfloat16", "bfloat16"), ("float32", "float32")])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("count", [49, 65, 128, 129, 4099])
def test_table_equals_launches_of_a_few(env, p_dtype, g_dtype, bits, count):
    """One launch from the device table, each tensor as in a group of few."""
    torch, q, dev = env
    sizes = [(613 * i) % 2111 for i in range(count)]  # (the first is empty)
    d = tensors(torch, dev, sizes, getattr(torch, p_dtype), getattr(torch, g_dtype), bits, p_dtype == "float32", 6)
    few = clone(d)
    print(f"adamw table {count} {p_dtype} {g_dtype} {bits}", flush=True)
    whole = q.AdamWGroup(**d)
    assert (whole._device_table is not None) == (count > 49)
    q.nvfp4_adamw(whole, 2, **HYPER)
    for i in range(0, count, 40):
        q.nvfp4_adamw(q.AdamWGroup(**{k: None if v is None else v[i:i + 40] for k, v in few.items()}), 2, **HYPER)
    torch.cuda.synchronize()
    for k, v in d.items():
        if v is not None:
            for i, t in enumerate(v):
                assert t is None or torch.equal(t.view(torch.uint8), few[k][i].view(torch.uint8)), f"{k} of tensor {i}"


@pytest.mark.parametrize("bits", [32, 8])
def test_table_of_large_tensors_and_a_captured_graph(env, bits):
    torch, q, dev = env
    count = 49 if bits == 32 else 98
    sizes = [1_000_003 if bits == 32 else 400_003] * count
    d = tensors(torch, dev, sizes, torch.float32, torch.float32, bits, False, 7)
    few = clone(d)
    print(f"adamw large table {bits}", flush=True)
    whole, parts = q.AdamWGroup(**d), [q.AdamWGroup(**{k: None if v is None else v[i:i + 7] for k, v in few.items()})
                                       for i in range(0, count, 7)]
    assert whole._device_table is not None
    q.nvfp4_adamw(whole, 1, **HYPER)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.nvfp4_adamw(whole, 2, **HYPER)
    for p in parts:
        q.nvfp4_adamw(p, 1, **HYPER)
    for i in range(3):
        graph.replay()
        for p in parts:
            q.nvfp4_adamw(p, 2, **HYPER)
        torch.cuda.synchronize()
        for k in ("params", "m", "v"):
            for a, b in zip(d[k], few[k]):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), f"replay {i}: {k}"


def test_another_stream_and_a_captured_graph(env):
    torch, q, dev = env
    for bits in (32, 8):
        d = tensors(torch, dev, [1000, 129, 5000], torch.float32, torch.float32, bits, True, 4)
        eager, side = clone(d), torch.cuda.Stream()
        grp, egrp = q.AdamWGroup(**d), q.AdamWGroup(**eager)
        torch.cuda.synchronize()
        q.nvfp4_adamw(grp, 2, stream=side, **HYPER)
        side.synchronize()
        q.nvfp4_adamw(egrp, 2, **HYPER)
        graph = torch.cuda.CUDAGraph()
        print(f"adamw capture bits {bits}", flush=True)
        with torch.cuda.graph(graph):
            q.nvfp4_adamw(grp, 3, **HYPER)
        for i in range(3):
            for a, b in zip(d["grads"], eager["grads"]):
                a.copy_(b.mul_(-0.7))
            graph.replay()
            q.nvfp4_adamw(egrp, 3, **HYPER)
            torch.cuda.synchronize()
            for k in ("params", "m", "v", "copies"):
                for a, b in zip(d[k], eager[k]):
                    assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), f"replay {i}: {k}"


def test_refuses_tensors_that_do_not_fit(env):
    torch, q, dev = env
    f, b = torch.zeros(256, device=dev), torch.zeros(256, device=dev, dtype=torch.bfloat16)
    e, s = torch.zeros(256, device=dev, dtype=torch.uint8).view(torch.float8_e4m3fn), torch.zeros(2, device=dev)
    q.AdamWGroup([f], [b], [f], [f], copies=[b])
    q.AdamWGroup([f], [b], [e], [e], [s], [s])
    for args, err in [(([f], [f[:255]], [f], [f]), ValueError), (([f], [f], [b], [f]), TypeError),
                      (([f], [f], [e], [e]), TypeError), (([f], [f], [f], [f], [s], [s]), TypeError),
                      (([f], [f], [e], [e], [s[:1]], [s]), ValueError), (([f, f], [f, b], [f, f], [f, f]), TypeError),
                      (([f, b], [f, f], [f, f], [f, f]), TypeError), (([f[::2]], [f[::2]], [f[::2]], [f[::2]]), ValueError),
                      (([b], [f], [f], [f], None, None, [b]), ValueError), (([f], [f], [f], [f], None, None, [f]), TypeError),
                      (([f], [f.cpu()], [f], [f]), TypeError), (([f, f], [f, f], [f, f], [f, f]), ValueError)]:
        with pytest.raises(err):
            q.AdamWGroup(*args)
    grp = q.AdamWGroup([f], [f.clone()], [f.clone()], [f.clone()])
    for bad in (dict(step=0, lr=1e-3), dict(step=1, lr=float("nan")), dict(step=1, lr=1e-3, beta1=1.0)):
        with pytest.raises(RuntimeError):
            q.nvfp4_adamw(grp, **bad)
    with pytest.raises(TypeError):
        q.nvfp4_adamw(grp, 1, 1e-3, grad_scale=s)
    with pytest.raises(ValueError):
        q.nvfp4_adamw(grp, 1, 1e-3, grad_scale=torch.ones(1))


@pytest.mark.parametrize("bits", [32, 8])
def test_a_large_step_equals_its_parts(env, bits):
    """A launch that moves more than the caches hold, against the same
    elements in groups of their own that the caches do hold."""
    torch, q, dev = env
    n, part = 50_000_000, 128 * 1000
    d = tensors(torch, dev, [n, 77], torch.float32, torch.float32, bits, True, 6)
    cuts = [(s, s + part) for s in (0, 128 * 100000, (n - part) // 128 * 128)]

    def cut(k, t, s, e):
        return t[s // 128:e // 128].clone() if k.endswith("scales") else t[s:e].clone()
    small = [{k: None if v is None else [cut(k, v[0], s, e)] for k, v in d.items()} for s, e in cuts]
    print(f"adamw large bits {bits}", flush=True)
    q.nvfp4_adamw(q.AdamWGroup(**d), 9, **HYPER)
    for (s, e), one in zip(cuts, small):
        q.nvfp4_adamw(q.AdamWGroup(**one), 9, **HYPER)
        for k, v in one.items():
            if v is not None and k != "grads":
                assert torch.equal(v[0].view(torch.uint8), cut(k, d[k][0], s, e).view(torch.uint8)), k


def test_offsets_past_32_bits(env):
    """A tensor of more than 2^32 elements in 8 bits: its ends as if alone."""
    torch, q, dev = env
    n, part = 2 ** 32 + 128 * 9 + 5, 128 * 50
    p = torch.zeros(n, dtype=torch.bfloat16, device=dev)
    g = torch.zeros(n, dtype=torch.bfloat16, device=dev)
    tail = (n - part) // 128 * 128
    gen = torch.Generator(device=dev)
    gen.manual_seed(8)
    for s, e in ((0, part), (tail, n)):
        p[s:e] = torch.randn(e - s, generator=gen, device=dev).bfloat16()
        g[s:e] = torch.randn(e - s, generator=gen, device=dev).bfloat16()
    grp = q.AdamWGroup.with_states([p], [g], bits=8)
    small = [q.AdamWGroup.with_states([p[s:e].clone()], [g[s:e].clone()], bits=8) for s, e in ((0, part), (tail, n))]
    print("adamw past 32 bits", flush=True)
    for step in (1, 2):
        for x in [grp] + small:
            q.nvfp4_adamw(x, step, **HYPER)
    torch.cuda.synchronize()
    for (s, e), x in zip(((0, part), (tail, n)), small):
        assert torch.equal(p[s:e], x.params[0])
        for a, b in ((grp.m[0], x.m[0]), (grp.v[0], x.v[0])):
            assert torch.equal(a[s:e].view(torch.uint8), b.view(torch.uint8))
        for a, b in ((grp.m_scales[0], x.m_scales[0]), (grp.v_scales[0], x.v_scales[0])):
            assert torch.equal(a[s // 128:][: b.numel()], b)
