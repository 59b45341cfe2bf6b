"""The example's gradient clipping (examples/expert_layer.py), on the CPU."""
import math
import os
import sys

import pytest
import torch

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
