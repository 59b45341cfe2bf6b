"""The training-step driver's layer of experts, the example's gradient clipping
(examples/expert_layer.py) and the search for overlaps among an AdamWGroup's
buffers, on the CPU."""
import math
import os
import sys

import pytest
import torch

import quantize_precision_gemm_amd as q

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_the_example_leaves_a_step_out_whose_gradients_are_not_finite(value):
    """The factor of a norm that is not finite is not finite itself: the AdamW
    step then writes nothing (a factor of 0 would make NaN of an infinity)."""
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import expert_layer
    g = torch.full((50,), 0.25)
    assert expert_layer.clip_factor([g], 10.0).item() == 1.0
    big = expert_layer.clip_factor([g, 16 * g], 0.5).item()
    # one division, a root and 101 sums of exact squares: 104 roundings of 2^-24 at most
    assert abs(big * 0.25 * math.sqrt(50 * 257) / 0.5 - 1) <= 104 * 2.0 ** -24
    g[7] = value
    assert not math.isfinite(expert_layer.clip_factor([g], 10.0).item())


class Recorder:
    """Stands in for the package: the calls a layer makes, and their workspaces."""
    FPROP, DGRAD, WGRAD = q.FPROP, q.DGRAD, q.WGRAD
    need = {q.FPROP: 48, q.DGRAD: 1 << 20, q.WGRAD: 0}

    def __init__(self):
        self.calls = []

    def nvfp4_bf16_grouped_gemm_workspace(self, pass_, E, T, N, K):
        assert (E, T, N, K) == (2, 6, 16, 24)
        return self.need[pass_]

    def nvfp4_bf16_grouped_gemm(self, pass_, a, b, ends, out_dtype=None, out=None, workspace=None, stream=None):
        self.calls.append((pass_, workspace))


def test_a_layer_of_experts_holds_its_workspaces():
    """One for each pass (dgrad and wgrad run beside each other), the same in
    every step."""
    from quantize_precision_gemm_amd.step import BF16Experts
    r = Recorder()
    bf16 = torch.bfloat16
    layer = BF16Experts(r, torch, torch.zeros(6, 24, dtype=bf16), torch.zeros(2, 16, 24, dtype=bf16),
                        torch.zeros(6, 16, dtype=bf16), torch.zeros(2, dtype=torch.int32))
    for _ in range(2):
        for _, op in layer.forward_ops() + layer.dgrad_ops() + layer.wgrad_ops():
            op()
    assert [p for p, _ in r.calls] == [q.FPROP, q.DGRAD, q.WGRAD] * 2
    for p, ws in r.calls:
        assert ws is not None and ws.dtype == torch.uint8 and ws.dim() == 1 and ws.numel() == r.need[p]
    assert all(r.calls[i][1] is r.calls[i + 3][1] for i in range(3))
    assert r.calls[0][1].data_ptr() != r.calls[1][1].data_ptr()


@pytest.mark.parametrize("written,read,found", [
    ([], [], False),
    ([(0, 16)], [(0, 16)], True),
    ([(0, 16), (16, 32)], [(32, 48), (32, 48)], False),            # neighbours; gradients may be shared
    ([(0, 16), (12, 20)], [], True),
    ([(40, 48), (0, 100)], [], True),                              # one inside another
    ([(0, 16), (64, 80)], [(20, 60), (10, 11)], True),
    ([(0, 16), (64, 80)], [(20, 60), (16, 64)], False),
    ([(0, 16), (64, 80)], [(80, 96), (8, 100)], True),
    ([(8, 8), (0, 16)], [(12, 12)], False),                        # tensors without elements
    ([(0, 4), (4, 8), (8, 12), (11, 16)], [], True),
    ([(100, 200)], [(0, 50), (20, 101)], True),
    ([(100, 200)], [(0, 300), (10, 20)], True),
])
def test_overlaps_of_written_buffers(written, read, found):
    for w in (written, written[::-1]):
        for r in (read, read[::-1]):
            assert q._overlapping(w, r) == found
