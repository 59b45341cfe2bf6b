"""GPU tests of rows that are not finite in the int8 row quantiser
(nvfp4_i8_quantize) and of their products."""
import pytest

from tests.gpu_util import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    ensure_built()
    import quantize_precision_gemm_amd as q
    return torch, q, torch.device("cuda:0")


@pytest.mark.parametrize("cols", [32, 1024, 2048, 8208, 20480])
def test_int8_rows_that_are_not_finite(env, cols):
    """Their scale is their largest magnitude / 127 (infinity or NaN), their codes
    are 0 and their products NaN; the other rows are as without them."""
    torch, q, dev = env
    g = torch.Generator(device=dev)
    g.manual_seed(cols)
    for rows in (9, 700):
        x = torch.randn(rows, cols, generator=g, device=dev).bfloat16()
        want = q.nvfp4_i8_quantize(x)
        inf, nan = float("inf"), float("nan")
        bad = {1: [inf], 3: [-inf], 4: [nan], 6: [nan, inf, -nan, -inf]}
        for r, values in bad.items():
            for i, value in enumerate(values):
                x[r, (7 * i + cols - 3) % cols] = value
        print(f"i8 not finite {rows} x {cols}", flush=True)
        got = q.nvfp4_i8_quantize(x)
        keep = torch.ones(rows, dtype=torch.bool, device=dev)
        keep[list(bad)] = False
        assert torch.equal(got.codes[keep], want.codes[keep]) and torch.equal(got.scales[keep], want.scales[keep])
        assert not got.codes[~keep].any().item()
        assert torch.isinf(got.scales[[1, 3]]).all().item() and (got.scales[[1, 3]] > 0).all().item()
        assert torch.isnan(got.scales[[4, 6]]).all().item()
        y = q.nvfp4_i8_gemm(got, q.nvfp4_i8_quantize(torch.ones(24, cols, device=dev).bfloat16()))
        assert torch.isnan(y[~keep]).all().item() and torch.isfinite(y[keep]).all().item()
