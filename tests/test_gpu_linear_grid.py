"""A linear layer of a few rows and so many columns that tiles of 64 columns by 8
waves would not fit into one grid.  Whole numbers, whose sums bf16 holds: the product's bits."""
import pytest
import torch

import quantize_precision_gemm_amd as q

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_more_columns_than_a_grid_of_wide_tiles():
    T, N, K = 16, 180_000_000, 8
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    x = torch.randint(-4, 5, (T, K), generator=g, device=DEV, dtype=torch.bfloat16)
    w = torch.randint(-4, 5, (N, K), generator=g, device=DEV, dtype=torch.bfloat16)
    out = torch.full((T, N), 300.0, dtype=torch.bfloat16, device=DEV)
    q.nvfp4_bf16_linear(x, w, out=out)
    step = 20_000_000
    for n in range(0, N, step):
        want = torch.zeros(T, step, device=DEV)
        for k in range(K):
            want += x[:, k, None].float() * w[n:n + step, k].float()
        assert torch.equal(out[:, n:n + step].float(), want), n
