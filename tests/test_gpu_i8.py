"""GPU tests of the int8 row quantiser and product (nvfp4_i8_quantize,
nvfp4_i8_gemm).

The codes equal those of exact arithmetic: 127 x / amax in 64 bits is never
nearer to a tie than 2^-16 of its value unless it is one, and both round ties
to even.  A scale is one division: half a step, 2^-24.
The sum is exact; its conversion and the two products with scales are three
roundings: |c - exact| <= 3.01 * 2^-24 |exact|, and a bf16 output is off by
2^-8 of the value more.
"""
import pytest

from tests.gpu_util import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    ensure_built()
    import quantize_precision_gemm_amd as q
    return torch, q, torch.device("cuda:0")


def exact_codes(torch, x):
    x = x.double()
    amax = x.abs().amax(1)
    return torch.round(127.0 * x / torch.where(amax > 0, amax, 1.0)[:, None]).to(torch.int8), amax / 127.0


def check_quant(torch, q, x, what):
    print(f"i8 quantize {what}", flush=True)
    got = q.nvfp4_i8_quantize(x)
    torch.cuda.synchronize()
    codes, scales = exact_codes(torch, x)
    assert torch.equal(got.codes, codes), what
    assert ((got.scales.double() - scales).abs() <= 2.0 ** -24 * scales + 2.0 ** -150).all().item(), what
    return got


@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 32), (7, 2048), (2, 2064), (5, 4096), (1, 5120), (33, 8192),
                                       (2, 20480), (4, 24592), (257, 1296), (1, 131056)])
def test_quantize(env, rows, cols):
    torch, q, dev = env
    g = torch.Generator(device=dev)
    g.manual_seed(rows * 7 + cols)
    x = torch.randn(rows, cols, generator=g, device=dev) * torch.exp(2 * torch.randn(rows, 1, generator=g, device=dev))
    check_quant(torch, q, x.bfloat16(), f"{rows} x {cols}")


def test_quantize_ties_and_extremes(env):
    torch, q, dev = env
    rows = []
    half = torch.arange(-254, 255, 2, device=dev).float() / 2  # 255 codes
    for top in (127.0, 254.0, 2.0 ** 100, 2.0 ** -100, 2.0 ** -126, 2.0 ** -133 * 127, 3.3895313892515355e38):
        x = torch.zeros(512, device=dev)
        x[:255] = half * (top / 127.0)
        x[255:509] = (torch.arange(-127, 127, device=dev).float() + 0.5) * (top / 127.0)  # ties, where bf16 holds them
        x[509], x[510], x[511] = top, -top, top / 2
        rows.append(x)
    rows.append(torch.zeros(512, device=dev))
    rows.append(-torch.zeros(512, device=dev))
    x = torch.stack(rows).bfloat16()
    got = check_quant(torch, q, x, "ties and extremes")
    assert got.scales[-1].item() == 0.0 and got.scales[-2].item() == 0.0


def test_every_pair_of_significands(env):
    """All quotients of 8-bit significands over the exponents that give a code."""
    torch, q, dev = env
    sig = torch.arange(128, 256, device=dev).double()
    rows = []
    for shift in range(0, 9):
        rows.append((sig * 2.0 ** -shift)[None].expand(128, 128))
    x = torch.cat(rows, 1)                                     # 128 rows, 9 x 128 columns
    x = torch.where(x <= sig[:, None], x, -x / 2)              # none above the row's maximum
    x = torch.cat([x, sig[:, None].expand(128, 16)], 1).bfloat16()
    check_quant(torch, q, x, "significands")


def test_quantize_padded(env):
    torch, q, dev = env
    buf = torch.full((9, 80), float("nan"), dtype=torch.bfloat16, device=dev)
    x = buf[:, :48]
    x.copy_(torch.randn(9, 48, device=dev))
    codes = torch.full((9, 96), 99, dtype=torch.int8, device=dev)
    out = q.I8Tensor(codes[:, :48], torch.empty(9, device=dev))
    print("i8 quantize padded", flush=True)
    q.nvfp4_i8_quantize(x, out=out)
    want, _ = exact_codes(torch, x)
    assert torch.equal(out.codes, want)
    assert (codes[:, 48:] == 99).all().item()
    empty = q.nvfp4_i8_quantize(torch.empty(0, 32, dtype=torch.bfloat16, device=dev))
    assert tuple(empty.shape) == (0, 32)
    none = q.nvfp4_i8_quantize(torch.empty(3, 0, dtype=torch.bfloat16, device=dev))
    assert not none.scales.any().item()


def problem(torch, dev, M, N, K, seed, full=False):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def codes(r):
        return torch.randint(-128 if full else -127, 128, (r, K), generator=g, device=dev).to(torch.int8)
    a, b = codes(M), codes(N)
    sa = torch.exp(torch.randn(M, generator=g, device=dev)) * 0.01
    sb = torch.exp(torch.randn(N, generator=g, device=dev)) * 0.003
    return a, sa, b, sb


def check_gemm(torch, got, a, sa, b, sb, what):
    want = (a.double() @ b.double().t()) * sa.double()[:, None] * sb.double()[None]
    tol = 3.01 * 2.0 ** -24 * want.abs()
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (want.abs() + tol)
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any().item(), f"{what}: {int(bad.sum())} elements off, first at {bad.nonzero()[0].tolist()}"


@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (1, 3, 32), (1, 4096, 5120), (1, 333, 1296), (2, 64, 128), (7, 130, 208),
                                   (16, 5003, 1296), (17, 256, 64), (31, 65, 2048), (33, 4100, 576), (64, 512, 640),
                                   (65, 100, 144), (127, 129, 1040), (128, 256, 512), (200, 1000, 272), (255, 257, 400),
                                   (256, 256, 128), (257, 513, 112), (300, 520, 1296), (777, 1288, 640), (1100, 72, 3088),
                                   (520, 2056, 16),
                                   (5000, 2568, 2064), (7900, 2568, 1040), (48, 512, 4112)])
def test_gemm(env, M, N, K):
    torch, q, dev = env
    a, sa, b, sb = problem(torch, dev, M, N, K, M + N + K)
    for dt in (torch.float32, torch.bfloat16):
        print(f"i8 gemm {M} {N} {K} {dt}", flush=True)
        got = q.nvfp4_i8_gemm(q.I8Tensor(a, sa), q.I8Tensor(b, sb), dt)
        torch.cuda.synchronize()
        assert got.dtype == dt and tuple(got.shape) == (M, N)
        check_gemm(torch, got, a, sa, b, sb, f"{M} {N} {K} {dt}")
        assert torch.equal(got, q.nvfp4_i8_gemm(q.I8Tensor(a, sa), q.I8Tensor(b, sb), dt))


@pytest.mark.parametrize("M,N", [(3, 20), (300, 264)])
def test_longest_sums_do_not_overflow(env, M, N):
    torch, q, dev = env
    K = (1 << 17) - 16
    a = torch.full((M, K), -128, dtype=torch.int8, device=dev)
    b = torch.full((N, K), -128, dtype=torch.int8, device=dev)
    b[1] = 127
    one = torch.ones(max(M, N), device=dev)
    print(f"i8 gemm longest {M} {N}", flush=True)
    got = q.nvfp4_i8_gemm(q.I8Tensor(a, one[:M]), q.I8Tensor(b, one[:N]), torch.float32)
    torch.cuda.synchronize()
    check_gemm(torch, got, a, one[:M], b, one[:N], "longest")


@pytest.mark.parametrize("M,N,K", [(5, 37, 96), (290, 301, 176)])
def test_gemm_padded(env, M, N, K):
    torch, q, dev = env
    a, sa, b, sb = problem(torch, dev, M, N, K, 5, full=True)

    def padded(x):
        buf = torch.full((x.shape[0] + 1, K + 48), 77, dtype=torch.int8, device=dev)
        buf[: x.shape[0], :K] = x
        return buf[: x.shape[0], :K]
    for dt in (torch.float32, torch.bfloat16):
        buf = torch.full((M + 2, (N + 3) // 4 * 4 + 8), -7.0, dtype=dt, device=dev)
        print(f"i8 gemm padded {M} {N} {K} {dt}", flush=True)
        q.nvfp4_i8_gemm(q.I8Tensor(padded(a), sa), q.I8Tensor(padded(b), sb), out=buf[:M, :N])
        torch.cuda.synchronize()
        check_gemm(torch, buf[:M, :N], a, sa, b, sb, "padded")
        assert (buf[M:] == -7.0).all().item() and (buf[:, N:] == -7.0).all().item()


def test_empty_products(env):
    torch, q, dev = env
    def t(r, k):
        return q.I8Tensor(torch.ones(r, k, dtype=torch.int8, device=dev), torch.ones(r, device=dev))
    print("i8 gemm empty", flush=True)
    assert tuple(q.nvfp4_i8_gemm(t(0, 32), t(5, 32)).shape) == (0, 5)
    assert tuple(q.nvfp4_i8_gemm(t(4, 32), t(0, 32)).shape) == (4, 0)
    for M in (3, 300):
        out = torch.full((M, 8), 5.0, device=dev)
        q.nvfp4_i8_gemm(t(M, 0), t(8, 0), out=out)
        assert not out.any().item()


@pytest.mark.parametrize("M", [4, 300])
def test_scales_that_are_not_finite_stay_in_their_row_and_column(env, M):
    torch, q, dev = env
    N = 48
    a, sa, b, sb = problem(torch, dev, M, N, 64, 8)
    clean = q.nvfp4_i8_gemm(q.I8Tensor(a, sa.clone()), q.I8Tensor(b, sb.clone()), torch.float32)
    sa[2], sb[7] = float("nan"), float("nan")
    print("i8 gemm NaN scales", flush=True)
    got = q.nvfp4_i8_gemm(q.I8Tensor(a, sa), q.I8Tensor(b, sb), torch.float32)
    keep = (torch.arange(M, device=dev) != 2)[:, None] & (torch.arange(N, device=dev) != 7)[None]
    assert torch.equal(got[keep], clean[keep])
    assert torch.isnan(got[2]).all().item() and torch.isnan(got[:, 7]).all().item()


def test_linear_layer_in_int8(env):
    """Quantise, multiply: each factor is off by half a code, scale / 2."""
    torch, q, dev = env
    M, N, K = 37, 264, 640
    g = torch.Generator(device=dev)
    g.manual_seed(6)
    x, w = torch.randn(M, K, generator=g, device=dev).bfloat16(), torch.randn(N, K, generator=g, device=dev).bfloat16()
    print("i8 linear", flush=True)
    xq, wq = q.nvfp4_i8_quantize(x), q.nvfp4_i8_quantize(w)
    y = q.nvfp4_i8_gemm(xq, wq, torch.float32).double()
    ex, ew = xq.scales.double()[:, None] / 2, wq.scales.double()[:, None] / 2
    xd, wd = x.double(), w.double()
    bound = xd.abs() @ ew.expand(N, K).t() + ex * wd.abs().sum(1)[None] + K * ex * ew.t()
    assert ((y - xd @ wd.t()).abs() <= 1.001 * bound).all().item()


def test_another_stream_and_a_captured_graph(env):
    torch, q, dev = env
    for M in (1, 40, 300):
        x, w = torch.randn(M, 640, device=dev).bfloat16(), torch.randn(264, 640, device=dev).bfloat16()
        wq = q.nvfp4_i8_quantize(w)
        want = q.nvfp4_i8_gemm(q.nvfp4_i8_quantize(x), wq)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        got = q.nvfp4_i8_gemm(q.nvfp4_i8_quantize(x, stream=side), wq, stream=side)
        side.synchronize()
        assert torch.equal(got, want)
        xq, out = q.nvfp4_i8_quantize(x), torch.zeros_like(want)
        graph = torch.cuda.CUDAGraph()
        print(f"i8 capture {M}", flush=True)
        with torch.cuda.graph(graph):
            q.nvfp4_i8_quantize(x, out=xq)
            q.nvfp4_i8_gemm(xq, wq, out=out)
        for i in range(3):
            x.mul_(-0.5).add_(0.01)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, q.nvfp4_i8_gemm(q.nvfp4_i8_quantize(x), wq)), f"replay {i}"


def test_refuses_tensors_that_do_not_fit(env):
    torch, q, dev = env
    c, s = torch.zeros(4, 32, dtype=torch.int8, device=dev), torch.zeros(4, device=dev)
    a = q.I8Tensor(c, s)
    for bad, err in [(q.I8Tensor(c.float(), s), TypeError), (q.I8Tensor(c, s[:3]), ValueError),
                     (q.I8Tensor(c, s.double()), TypeError), (q.I8Tensor(c, s.cpu()), ValueError),
                     (q.I8Tensor(c.t(), torch.zeros(32, device=dev)), ValueError), (q.I8Tensor(c[:, :16], s), ValueError)]:
        with pytest.raises(err):
            q.nvfp4_i8_gemm(a, bad)
    with pytest.raises((TypeError, RuntimeError)):
        q.nvfp4_i8_gemm(a, a, torch.float16)
    with pytest.raises(ValueError):
        q.nvfp4_i8_gemm(a, a, out=torch.zeros(4, 5, device=dev))
    with pytest.raises(RuntimeError):  # rows that are not whole 16-byte pieces
        q.nvfp4_i8_gemm(q.I8Tensor(c[:, :24], s), q.I8Tensor(c[:, :24], s))
    with pytest.raises(ValueError):
        q.nvfp4_i8_quantize(torch.zeros(4, 32, dtype=torch.bfloat16, device=dev), out=q.I8Tensor(c[:3], s[:3]))


def test_offsets_past_32_bits(env):
    torch, q, dev = env
    N, K, far = 40, 96, 2 ** 22
    for M in (1100, 1300):
        a, sa, b, sb = problem(torch, dev, M, N, K, 4)
        wide = torch.empty(M, far, dtype=torch.int8, device=dev)[:, :K]
        wide.copy_(a)
        out = torch.empty(M, far // 2, dtype=torch.bfloat16, device=dev)[:, :N]
        print(f"i8 far {M}", flush=True)
        q.nvfp4_i8_gemm(q.I8Tensor(wide, sa), q.I8Tensor(b, sb), out=out)
        torch.cuda.synchronize()
        check_gemm(torch, out, a, sa, b, sb, "far")
        x = torch.randn(M, K, device=dev).bfloat16()
        far_x = torch.empty(M, far // 2, dtype=torch.bfloat16, device=dev)[:, :K]
        far_x.copy_(x)
        got = q.nvfp4_i8_quantize(far_x, out=q.I8Tensor(wide, torch.empty(M, device=dev)))
        want, _ = exact_codes(torch, x)
        assert torch.equal(got.codes, want)


def test_quantize_many_short_rows(env):
    """More rows than a launch has workgroups."""
    torch, q, dev = env
    g = torch.Generator(device=dev)
    g.manual_seed(3)
    rows = 4 * 2 ** 22 + 5
    x = torch.randn(rows, 16, generator=g, device=dev).bfloat16()
    print("i8 quantize many rows", flush=True)
    got = q.nvfp4_i8_quantize(x)
    torch.cuda.synchronize()
    for part in (slice(0, 100000), slice(rows - 100000, rows)):
        codes, scales = exact_codes(torch, x[part])
        assert torch.equal(got.codes[part], codes)
        assert ((got.scales[part].double() - scales).abs() <= 2.0 ** -24 * scales).all().item()
