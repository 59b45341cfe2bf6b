"""GPU tests of the products grouped by expert (nvfp4_bf16_grouped_gemm)
against the 64-bit product of the same bf16 operands, expert by expert.

Tolerance, from the arithmetic: products of two bf16 values are exact in
fp32; a sum of C of them takes C additions, each off by at most one unit in
the last place (2^-23 of a partial sum, which sum |a||b| bounds), and joining
the parts of a split contraction at most 8 more.  So
|c - exact| <= (C + 8) 2^-23 sum |a||b|, and a bf16 output is off by half a
step, 2^-8 |c|, more.
"""
import numpy as np
import pytest

from tests.gpu_util import ensure_built

pytestmark = pytest.mark.gpu

FPROP, DGRAD, WGRAD = 0, 1, 2


@pytest.fixture(scope="module")
def env():
    import torch
    ensure_built()
    import quantize_precision_gemm_amd as q
    return torch, q, torch.device("cuda:0")


def clamped(ends, T):
    """[begin, end) of each expert as the kernels read the ends."""
    out, last = [], 0
    for e in ends:
        e = max(last, min(max(int(e), 0), T))
        out.append((last, e))
        last = e
    return out


def ends_of(rows):
    return list(np.cumsum(rows))


def operands(torch, dev, pass_, T, E, N, K, seed):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def rnd(*s):
        return torch.randn(s, generator=g, device=dev).bfloat16()
    x, w, dy = rnd(T, K), rnd(E, N, K), rnd(T, N)
    return {FPROP: (x, w), DGRAD: (dy, w), WGRAD: (dy, x)}[pass_]


def reference(torch, pass_, a, b, ends, E):
    """(exact product, sum |a||b|, longest contraction) in 64 bits."""
    T = a.shape[0]
    spans = clamped(ends, T)
    if pass_ == WGRAD:
        want = torch.zeros(E, a.shape[1], b.shape[1], dtype=torch.float64, device=a.device)
        size = torch.zeros_like(want)
        for e, (s, t) in enumerate(spans):
            ra, rb = a[s:t].double(), b[s:t].double()
            want[e], size[e] = ra.t() @ rb, ra.abs().t() @ rb.abs()
        return want, size, max([t - s for s, t in spans] + [1])
    cols = b.shape[1] if pass_ == FPROP else b.shape[2]
    want = torch.zeros(T, cols, dtype=torch.float64, device=a.device)
    size = torch.zeros_like(want)
    for e, (s, t) in enumerate(spans):
        w = b[e].double()
        w = w.t() if pass_ == FPROP else w
        want[s:t], size[s:t] = a[s:t].double() @ w, a[s:t].double().abs() @ w.abs()
    return want, size, a.shape[1]


def check(torch, got, want, size, C, what):
    tol = (C + 8) * 2.0 ** -23 * size
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (want.abs() + tol)
    bad = ~((got.double() - want).abs() <= tol)  # a NaN is bad too
    assert not bad.any().item(), f"{what}: {int(bad.sum())} elements off, first at {bad.nonzero()[0].tolist()}"


CASES = [
    # rows of each expert, rows behind the last, N, K
    ([1], 0, 8, 8),
    ([0], 0, 16, 16),
    ([0, 0, 0], 5, 24, 40),
    ([1, 0, 2, 1], 0, 64, 128),
    ([3, 17, 0, 33, 16], 2, 72, 136),
    ([255, 1, 256, 0, 257], 3, 264, 328),
    ([130, 0, 70, 513], 0, 520, 192),
    ([2] * 65, 1, 40, 64),
    ([5, 0, 1] * 50, 0, 48, 72),
    ([300], 300, 256, 64),
    ([40, 24], 0, 8, 1032),
    ([700, 20, 1000], 0, 1288, 648),
    # whole and partial rounds of the largest tiles, in each pass
    ([3000, 0, 2690], 10, 2568, 2056),
    ([130] * 60, 0, 264, 2056),
    ([2600, 5100, 100], 0, 2056, 2568),
    # rows for the 16-, 32- and 64-row products, more of some than a tile holds
    ([16, 3, 20, 9], 0, 520, 4104),
    ([30, 32, 41, 25], 1, 264, 2056),
    ([64, 50, 100, 3], 0, 136, 1032),
]


@pytest.mark.parametrize("pass_", [FPROP, DGRAD, WGRAD])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_passes(env, pass_, case):
    torch, q, dev = env
    rows, tail, N, K = CASES[case]
    E, T = len(rows), sum(rows) + tail
    ends = torch.tensor(ends_of(rows), dtype=torch.int32, device=dev)
    a, b = operands(torch, dev, pass_, T, E, N, K, case)
    want, size, C = reference(torch, pass_, a, b, ends_of(rows), E)
    for dt in (torch.float32, torch.bfloat16):
        print(f"grouped pass {pass_} rows {rows[:6]} N {N} K {K} {dt}", flush=True)
        got = q.nvfp4_bf16_grouped_gemm(pass_, a, b, ends, dt)
        torch.cuda.synchronize()
        assert got.dtype == dt and tuple(got.shape) == tuple(want.shape)
        check(torch, got, want, size, C, f"pass {pass_}")
        again = q.nvfp4_bf16_grouped_gemm(pass_, a, b, ends, dt)
        assert torch.equal(got, again), "a second call gives other bits"


@pytest.mark.parametrize("pass_", [FPROP, DGRAD, WGRAD])
def test_no_tokens_and_no_experts(env, pass_):
    torch, q, dev = env
    print(f"grouped empty pass {pass_}", flush=True)
    a, b = operands(torch, dev, pass_, 0, 3, 16, 24, 0)
    got = q.nvfp4_bf16_grouped_gemm(pass_, a, b, torch.zeros(3, dtype=torch.int32, device=dev))
    assert tuple(got.shape) == {FPROP: (0, 16), DGRAD: (0, 24), WGRAD: (3, 16, 24)}[pass_]
    assert not got.any().item()
    a, b = operands(torch, dev, pass_, 5, 0, 16, 24, 0)
    got = q.nvfp4_bf16_grouped_gemm(pass_, a, b, torch.zeros(0, dtype=torch.int32, device=dev))
    assert tuple(got.shape) == {FPROP: (5, 16), DGRAD: (5, 24), WGRAD: (0, 16, 24)}[pass_]
    assert not got.any().item()


def test_an_empty_contraction_writes_zeros(env):
    torch, q, dev = env
    ends = torch.tensor([2, 5], dtype=torch.int32, device=dev)
    x, w = torch.empty(5, 0, dtype=torch.bfloat16, device=dev), torch.empty(2, 16, 0, dtype=torch.bfloat16, device=dev)
    out = torch.full((5, 16), 7.0, device=dev)
    print("grouped K 0", flush=True)
    q.nvfp4_bf16_grouped_gemm(q.FPROP, x, w, ends, out=out)
    assert not out.any().item()
    w = torch.empty(2, 0, 24, dtype=torch.bfloat16, device=dev)
    out = torch.full((5, 24), 7.0, device=dev)
    print("grouped N 0", flush=True)
    q.nvfp4_bf16_grouped_gemm(q.DGRAD, x, w, ends, out=out)
    assert not out.any().item()


@pytest.mark.parametrize("pass_", [FPROP, DGRAD, WGRAD])
@pytest.mark.parametrize("ends", [[7, 3, 40], [-5, 10, 2000000000], [60, 60, 60], [-2147483648, 2147483647, 0]])
def test_ends_out_of_order_or_range(env, pass_, ends):
    """Such ends count as the nearest that are in order and range."""
    torch, q, dev = env
    T, N, K = 45, 32, 48
    a, b = operands(torch, dev, pass_, T, 3, N, K, 5)
    want, size, C = reference(torch, pass_, a, b, ends, 3)
    print(f"grouped ends {ends} pass {pass_}", flush=True)
    got = q.nvfp4_bf16_grouped_gemm(pass_, a, b, torch.tensor(ends, dtype=torch.int32, device=dev), torch.float32)
    check(torch, got, want, size, C, f"ends {ends}")


@pytest.mark.parametrize("pass_", [FPROP, DGRAD, WGRAD])
@pytest.mark.parametrize("big", [False, True])
def test_padded_operands_and_output(env, pass_, big):
    """Leading dimensions, expert strides and outputs with room between the
    rows; the room is neither read into the result nor written."""
    torch, q, dev = env
    rows = [333, 0, 290, 400] if big else [9, 0, 20, 4]
    N, K = (296, 328) if big else (40, 56)
    E, T = len(rows), sum(rows)
    ends = torch.tensor(ends_of(rows), dtype=torch.int32, device=dev)
    a, b = operands(torch, dev, pass_, T, E, N, K, 9)
    want, size, C = reference(torch, pass_, a, b, ends_of(rows), E)

    def padded(x):
        shape = list(x.shape)
        shape[-1] += 24
        shape[-2] += 3
        buf = torch.full(shape, float("nan"), dtype=x.dtype, device=dev)
        view = buf[..., : x.shape[-2], : x.shape[-1]]
        view.copy_(x)
        return view
    for dt in (torch.float32, torch.bfloat16):
        shape = list(want.shape)
        shape[-1] += 12
        shape[-2] += 2
        buf = torch.full(shape, -7.0, dtype=dt, device=dev)
        out = buf[..., : want.shape[-2], : want.shape[-1]]
        print(f"grouped padded pass {pass_} big {big} {dt}", flush=True)
        q.nvfp4_bf16_grouped_gemm(pass_, padded(a), padded(b), ends, out=out)
        torch.cuda.synchronize()
        check(torch, out, want, size, C, "padded")
        mask = torch.ones_like(buf, dtype=torch.bool)
        mask[..., : want.shape[-2], : want.shape[-1]] = False
        assert (buf[mask] == -7.0).all().item(), "written outside the output"


@pytest.mark.parametrize("pass_", [FPROP, DGRAD, WGRAD])
@pytest.mark.parametrize("size", [20, 300])
def test_what_is_not_finite_stays_in_its_expert(env, pass_, size):
    """NaN and infinities in one expert's rows, in another's weight and in the
    rows of no expert reach no other expert's output."""
    torch, q, dev = env
    rows, tail, N, K = [size + 1, size, 0, size + 3, 7], 6, 64, 88
    E, T = len(rows), sum(rows) + tail
    ends = torch.tensor(ends_of(rows), dtype=torch.int32, device=dev)
    a, b = operands(torch, dev, pass_, T, E, N, K, 3)
    s = ends_of(rows)[0]
    clean = q.nvfp4_bf16_grouped_gemm(pass_, a, b, ends, torch.float32)
    a[s:s + size] = float("nan")       # all of expert 1
    a[T - tail:] = float("inf")        # rows of no expert
    if pass_ == WGRAD:
        b[s:s + size] = float("inf")
        b[T - tail:] = float("nan")
    else:
        b[2] = float("nan")            # the weight of the expert without rows
    print(f"grouped not finite pass {pass_} size {size}", flush=True)
    got = q.nvfp4_bf16_grouped_gemm(pass_, a, b, ends, torch.float32)
    torch.cuda.synchronize()
    if pass_ == WGRAD:
        keep = [0, 2, 3, 4]
        assert torch.equal(got[keep], clean[keep])
        assert torch.isnan(got[1]).all().item()
    else:
        assert torch.equal(got[:s], clean[:s]) and torch.equal(got[s + size:], clean[s + size:])
        assert torch.isnan(got[s:s + size]).all().item()
        assert not got[T - tail:].any().item()


def test_one_expert_is_the_layer_of_the_plain_gemm(env):
    torch, q, dev = env
    T, N, K = 384, 264, 520
    ends = torch.tensor([T], dtype=torch.int32, device=dev)
    for pass_ in (FPROP, DGRAD, WGRAD):
        a, b = operands(torch, dev, pass_, T, 1, N, K, 11)
        plain = q.nvfp4_bf16_gemm(pass_, a, b if pass_ == WGRAD else b[0], torch.float32)
        print(f"grouped against plain pass {pass_}", flush=True)
        got = q.nvfp4_bf16_grouped_gemm(pass_, a, b, ends, torch.float32)
        _, size, C = reference(torch, pass_, a, b, [T], 1)
        diff = (got.reshape(plain.shape).double() - plain.double()).abs()
        assert (diff <= 2 * (C + 8) * 2.0 ** -23 * size.reshape(plain.shape)).all().item()


def test_another_stream_and_a_captured_graph(env):
    torch, q, dev = env
    rows, N, K = [100, 0, 37, 160], 264, 136
    E, T = len(rows), sum(rows)
    ends = torch.tensor(ends_of(rows), dtype=torch.int32, device=dev)
    ops = {p: operands(torch, dev, p, T, E, N, K, 20 + p) for p in (FPROP, DGRAD, WGRAD)}
    want = {p: q.nvfp4_bf16_grouped_gemm(p, *ops[p], ends) for p in ops}
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = {p: q.nvfp4_bf16_grouped_gemm(p, *ops[p], ends, stream=side) for p in ops}
    side.synchronize()
    for p in ops:
        assert torch.equal(got[p], want[p])
    outs = {p: torch.zeros_like(want[p]) for p in ops}
    graph = torch.cuda.CUDAGraph()
    print("grouped capture", flush=True)
    with torch.cuda.graph(graph):
        for p in ops:
            q.nvfp4_bf16_grouped_gemm(p, *ops[p], ends, out=outs[p])
    for i in range(3):  # the routing is read at replay
        split = ends_of([T - 30 * (i + 1), 10 * (i + 1), 20 * (i + 1), 0])
        ends.copy_(torch.tensor(split, dtype=torch.int32, device=dev))
        for p in ops:
            outs[p].zero_()
        graph.replay()
        torch.cuda.synchronize()
        for p in ops:
            assert torch.equal(outs[p], q.nvfp4_bf16_grouped_gemm(p, *ops[p], ends)), f"replay {i} pass {p}"


SPLITS = {
    # rows of each expert, rows behind the last, N, K: few tiles, a long contraction
    FPROP: [([90, 0, 130], 5, 72, 4104), ([200], 0, 264, 8200), ([140, 3], 0, 1032, 4104)],
    DGRAD: [([90, 0, 130], 5, 4104, 72), ([200], 0, 8200, 264), ([140, 3], 0, 4104, 1032)],
    WGRAD: [([4097], 0, 200, 136), ([6000, 0, 1, 2999], 7, 264, 72), ([20, 9000], 300, 8, 1032)],
}


@pytest.mark.parametrize("pass_", [FPROP, DGRAD, WGRAD])
@pytest.mark.parametrize("case", range(3))
def test_split_contraction(env, pass_, case):
    """In parts with the workspace that the query names, whole without one or
    with too little; the parts' sums do not depend on what the workspace held,
    and the output's surroundings stay."""
    torch, q, dev = env
    rows, tail, N, K = SPLITS[pass_][case]
    E, T = len(rows), sum(rows) + tail
    ends = torch.tensor(ends_of(rows), dtype=torch.int32, device=dev)
    a, b = operands(torch, dev, pass_, T, E, N, K, 60 + case)
    want, size, C = reference(torch, pass_, a, b, ends_of(rows), E)
    need = q.nvfp4_bf16_grouped_gemm_workspace(pass_, E, T, N, K)
    assert need > 0
    for dt in (torch.float32, torch.bfloat16):
        results = []
        for fill, size_ws in ((0, need), (255, need), (255, need + 48), (255, need - 16), (255, 0)):
            print(f"grouped split pass {pass_} rows {rows} N {N} K {K} {dt} workspace {size_ws}", flush=True)
            buf = torch.full((size_ws + 64,), fill, dtype=torch.uint8, device=dev)  # 255: NaN
            shape = list(want.shape)
            shape[-1] += 12
            shape[-2] += 2
            held = torch.full(shape, -7.0, dtype=dt, device=dev)
            out = held[..., : want.shape[-2], : want.shape[-1]]
            q.nvfp4_bf16_grouped_gemm(pass_, a, b, ends, out=out, workspace=buf[:size_ws])
            torch.cuda.synchronize()
            check(torch, out, want, size, C, f"workspace {size_ws}")
            mask = torch.ones_like(held, dtype=torch.bool)
            mask[..., : want.shape[-2], : want.shape[-1]] = False
            assert (held[mask] == -7.0).all().item(), "written outside the output"
            assert (buf[size_ws:] == fill).all().item(), "written behind the workspace"
            assert size_ws >= need or (buf == fill).all().item(), "a workspace that is too small was used"
            results.append(out.clone())
        assert torch.equal(results[0], results[1]) and torch.equal(results[0], results[2])
        assert torch.equal(results[3], results[4])
        assert torch.equal(results[0], q.nvfp4_bf16_grouped_gemm(pass_, a, b, ends, dt))


def test_refuses_workspaces_that_do_not_fit(env):
    torch, q, dev = env
    a, b = operands(torch, dev, WGRAD, 2048, 1, 64, 64, 72)
    ends = torch.tensor([2048], dtype=torch.int32, device=dev)
    for bad in (torch.empty(1 << 20), torch.empty(1 << 20, dtype=torch.uint8), torch.empty(1 << 18, device=dev),
                torch.empty(2, 1 << 19, dtype=torch.uint8, device=dev)):
        with pytest.raises(ValueError):
            q.nvfp4_bf16_grouped_gemm(WGRAD, a, b, ends, workspace=bad)
    with pytest.raises(TypeError):
        q.nvfp4_bf16_grouped_gemm(WGRAD, a, b, ends, workspace=1 << 20)
    with pytest.raises(RuntimeError):
        q.nvfp4_bf16_grouped_gemm(WGRAD, a, b, ends, workspace=torch.empty(1 << 20, dtype=torch.uint8, device=dev)[8:])


def test_split_contraction_in_a_captured_graph(env):
    torch, q, dev = env
    T, E, N, K = 4096, 2, 136, 72
    a, b = operands(torch, dev, WGRAD, T, E, N, K, 71)
    ends = torch.tensor([1000, T], dtype=torch.int32, device=dev)
    assert q.nvfp4_bf16_grouped_gemm_workspace(WGRAD, E, T, N, K) > 0
    q.nvfp4_bf16_grouped_gemm(WGRAD, a, b, ends)
    out = torch.zeros(E, N, K, dtype=torch.bfloat16, device=dev)
    graph = torch.cuda.CUDAGraph()
    print("grouped split capture", flush=True)
    with torch.cuda.graph(graph):
        q.nvfp4_bf16_grouped_gemm(WGRAD, a, b, ends, out=out)
    for i in range(3):
        ends.copy_(torch.tensor([1500 * i, T - 100 * i], dtype=torch.int32, device=dev))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, q.nvfp4_bf16_grouped_gemm(WGRAD, a, b, ends)), f"replay {i}"


def test_gradients_are_those_of_the_forward_product(env):
    """dX and dW against central differences of sum(Y * dY): the product is
    linear in each operand, so a step of 1/2 in one element (exact in bf16 for
    these whole numbers) gives the derivative exactly."""
    torch, q, dev = env
    rows, N, K = [3, 0, 2], 8, 16
    T = sum(rows)
    g = torch.Generator(device=dev)
    g.manual_seed(1)

    def whole(*s):
        return torch.randint(-4, 5, s, generator=g, device=dev).bfloat16()
    x, w, dy = whole(T, K), whole(3, N, K), whole(T, N)
    ends = torch.tensor(ends_of(rows), dtype=torch.int32, device=dev)

    def loss(x_, w_):
        return (q.nvfp4_bf16_grouped_gemm(q.FPROP, x_, w_, ends, torch.float32).double() * dy.double()).sum().item()
    dx = q.nvfp4_bf16_grouped_gemm(q.DGRAD, dy, w, ends, torch.float32)
    dw = q.nvfp4_bf16_grouped_gemm(q.WGRAD, dy, x, ends, torch.float32)
    for t, k in [(0, 0), (2, 5), (3, 15), (4, 7)]:
        up, down = x.clone(), x.clone()
        up[t, k] += 0.5
        down[t, k] -= 0.5
        assert loss(up, w) - loss(down, w) == dx[t, k].item()
    for e, n, k in [(0, 0, 0), (0, 7, 3), (1, 2, 2), (2, 4, 15)]:
        up, down = w.clone(), w.clone()
        up[e, n, k] += 0.5
        down[e, n, k] -= 0.5
        assert loss(x, up) - loss(x, down) == dw[e, n, k].item()


def test_refuses_tensors_that_do_not_fit(env):
    torch, q, dev = env
    a, b = operands(torch, dev, FPROP, 8, 2, 16, 24, 0)
    ends = torch.tensor([4, 8], dtype=torch.int32, device=dev)
    for bad in (ends.long(), ends.cpu(), ends[None], torch.zeros(4, dtype=torch.int32, device=dev)[::2], ends[:1]):
        with pytest.raises(ValueError):
            q.nvfp4_bf16_grouped_gemm(q.FPROP, a, b, bad)
    with pytest.raises(ValueError):
        q.nvfp4_bf16_grouped_gemm(5, a, b, ends)
    with pytest.raises(ValueError):
        q.nvfp4_bf16_grouped_gemm(q.DGRAD, a, b, ends)  # 24 columns for N = 16
    with pytest.raises(ValueError):
        q.nvfp4_bf16_grouped_gemm(q.WGRAD, a, a[:4], ends)
    with pytest.raises(TypeError):
        q.nvfp4_bf16_grouped_gemm(q.FPROP, a, b[0], ends)
    with pytest.raises(TypeError):
        q.nvfp4_bf16_grouped_gemm(q.FPROP, a, b.float(), ends)
    with pytest.raises(TypeError):
        q.nvfp4_bf16_grouped_gemm(q.FPROP, a, b, ends, torch.float16)
    with pytest.raises(ValueError):
        q.nvfp4_bf16_grouped_gemm(q.FPROP, a, b, ends, out=torch.empty(8, 24, device=dev))
    with pytest.raises(ValueError):
        q.nvfp4_bf16_grouped_gemm(q.WGRAD, a, a, ends, out=torch.empty(2, 24, 16, device=dev))
    odd = torch.zeros(8, 20, dtype=torch.bfloat16, device=dev)
    with pytest.raises(ValueError):
        q.nvfp4_bf16_grouped_gemm(q.FPROP, odd, torch.zeros(2, 16, 20, dtype=torch.bfloat16, device=dev), ends)


def test_offsets_past_32_bits(env):
    """Operands and outputs whose last rows lie more than 4 GiB behind their first."""
    torch, q, dev = env
    N, K, T, far = 64, 72, 1100, 2 ** 21  # 1100 rows, 4 MiB apart
    ends = torch.tensor([40, 40, T], dtype=torch.int32, device=dev)
    for pass_ in (FPROP, DGRAD, WGRAD):
        a, b = operands(torch, dev, pass_, T, 3, N, K, 40)
        want, size, C = reference(torch, pass_, a, b, [40, 40, T], 3)
        wide = torch.empty(T, far, dtype=torch.bfloat16, device=dev)
        wide[:, : a.shape[1]] = a
        if pass_ == WGRAD:
            place = b
            out = torch.empty(3, N, far, dtype=torch.float32, device=dev)[:, :, :K]
        else:
            place = torch.empty(3, 2 ** 30, dtype=torch.bfloat16, device=dev)[:, : N * K].view(3, N, K)
            place.copy_(b)
            out = torch.empty(T, far, dtype=torch.float32, device=dev)[:, : want.shape[1]]
        print(f"grouped far pass {pass_}", flush=True)
        q.nvfp4_bf16_grouped_gemm(pass_, wide[:, : a.shape[1]], place, ends, out=out)
        torch.cuda.synchronize()
        check(torch, out, want, size, C, f"far pass {pass_}")
        del wide, place, out
