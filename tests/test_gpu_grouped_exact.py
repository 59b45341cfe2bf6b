"""GPU tests of the products grouped by expert (nvfp4_bf16_grouped_gemm) on
whole numbers, where every order of the sums gives the same value.

Operands from -8 to 8 and contractions of at most 2^16 - 1 elements: every
product and every partial sum is a whole number below 2^22, exact in fp32.
So an fp32 output has to equal the exact product, and a bf16 output that
product rounded once, to the nearest even: a product left out or counted twice,
or a partial sum in fewer bits, shows in any kernel, half tile or split.
The expert counts 63, 64 and 128 put the rows of no expert on the last lane of
the search's first 64, alone behind them, and behind the second 64.
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


def operands(torch, dev, pass_, T, E, N, K, seed):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def whole(*s):
        return torch.randint(-8, 9, s, generator=g, device=dev).bfloat16()
    x, w, dy = whole(T, K), whole(E, N, K), whole(T, N)
    return {FPROP: (x, w), DGRAD: (dy, w), WGRAD: (dy, x)}[pass_]


def exact(torch, pass_, a, b, rows):
    """The product in 64 bits, expert by expert; zeros for rows of no expert."""
    parts, s = [], 0
    for e, n in enumerate(rows):
        ra = a[s:s + n].double()
        if pass_ == WGRAD:
            parts.append(ra.t().contiguous() @ b[s:s + n].double())
        else:
            w = b[e].double()
            parts.append(ra @ (w.t().contiguous() if pass_ == FPROP else w))
        s += n
    if pass_ == WGRAD:
        return torch.stack(parts)
    parts.append(torch.zeros(a.shape[0] - s, parts[0].shape[1], dtype=torch.float64, device=a.device))
    return torch.cat(parts)


CASES = [
    # rows of each expert, rows behind the last, N, K
    ([1, 0, 2, 1], 0, 64, 128),
    ([3, 17, 0, 33, 16], 2, 72, 136),
    ([255, 1, 256, 0, 257], 3, 264, 328),
    ([700, 20, 1000], 0, 1288, 648),
    ([3000, 0, 2690], 10, 2568, 2056),     # whole and partial rounds of the largest tiles, halves
    ([130] * 60, 0, 264, 2056),
    ([2600, 5100, 100], 0, 2056, 2568),
    ([16, 3, 20, 9], 0, 520, 4104),        # 16-, 32- and 64-row products
    ([30, 32, 41, 25], 1, 264, 2056),
    ([64, 50, 100, 3], 0, 136, 1032),
    ([1, 0, 3] * 21, 5, 40, 72),           # 63 experts
    ([2, 1] * 32, 3, 40, 72),              # 64
    ([1, 0, 2, 5] * 32, 7, 48, 64),        # 128
    ([40] * 63, 9, 264, 136),
    ([0] * 63 + [300], 40, 264, 136),
    ([7] * 127 + [200], 130, 520, 264),
    ([0] * 128, 33, 64, 64),
]


@pytest.mark.parametrize("pass_", [FPROP, DGRAD, WGRAD])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_whole_numbers(env, pass_, case):
    torch, q, dev = env
    rows, tail, N, K = CASES[case]
    E, T = len(rows), sum(rows) + tail
    ends = torch.tensor(np.cumsum(rows), dtype=torch.int32, device=dev)
    a, b = operands(torch, dev, pass_, T, E, N, K, case)
    want = exact(torch, pass_, a, b, rows).float()
    for dt in (torch.float32, torch.bfloat16):
        print(f"grouped whole numbers pass {pass_} experts {E} rows {T} N {N} K {K} {dt}", flush=True)
        got = q.nvfp4_bf16_grouped_gemm(pass_, a, b, ends, dt)
        assert torch.equal(got, want.to(dt))


SPLITS = {
    FPROP: [([90, 0, 130], 5, 72, 4104), ([200], 0, 264, 8200), ([60] * 64, 3, 72, 8200), ([0, 60] * 40, 2, 72, 8200)],
    DGRAD: [([90, 0, 130], 5, 4104, 72), ([200], 0, 8200, 264), ([1] * 64, 3, 4104, 72), ([0, 2] * 40, 2, 8200, 64)],
    WGRAD: [([4097], 0, 200, 136), ([6000, 0, 1, 2999], 7, 264, 72), ([20, 9000], 300, 8, 1032),
            ([5000] * 50 + [0] * 14, 11, 120, 128)],
}


@pytest.mark.parametrize("pass_", [FPROP, DGRAD, WGRAD])
@pytest.mark.parametrize("case", range(4))
def test_whole_numbers_in_parts(env, pass_, case):
    """With the workspace of a split contraction and without it."""
    torch, q, dev = env
    rows, tail, N, K = SPLITS[pass_][case]
    E, T = len(rows), sum(rows) + tail
    need = q.nvfp4_bf16_grouped_gemm_workspace(pass_, E, T, N, K)
    assert need > 0
    ends = torch.tensor(np.cumsum(rows), dtype=torch.int32, device=dev)
    a, b = operands(torch, dev, pass_, T, E, N, K, 50 + case)
    want = exact(torch, pass_, a, b, rows).float()
    for dt in (torch.float32, torch.bfloat16):
        for size in (need, 0):
            print(f"grouped whole numbers in parts pass {pass_} experts {E} {dt} workspace {size}", flush=True)
            ws = torch.full((size,), 255, dtype=torch.uint8, device=dev)
            got = q.nvfp4_bf16_grouped_gemm(pass_, a, b, ends, dt, workspace=ws)
            assert torch.equal(got, want.to(dt))
