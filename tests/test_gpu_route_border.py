"""Routing where values that the fast comparison cannot tell apart lie on both
sides of the border between the chosen and the others, more than two of them: equal ones
among the chosen and the next, and a larger one beyond.  And groups whose sums
of two pass fp32's range.  Against the definition in 64 bits, as
test_gpu_route.py has it (experts and places equal, weights within its tolerance)."""
import pytest
import torch

import quantize_precision_gemm_amd as q
from tests.test_gpu_route import DEV, check, randn

pytestmark = pytest.mark.gpu
LOWEST = torch.finfo(torch.float32).min
SIZES = [16, 33, 64, 128, 256, 320, 1024]  # the variants: lanes a row, experts a lane
SCORES = pytest.mark.parametrize("score", [q.SOFTMAX, q.SIGMOID])


def permuted(logits, seed):
    """Each row's experts in an order of its own, but for the first row's."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    order = torch.rand(logits.shape, generator=g, device=DEV).argsort(1)
    order[0] = torch.arange(logits.shape[1], device=DEV)
    return logits.gather(1, order)


@SCORES
@pytest.mark.parametrize("E", SIZES)
@pytest.mark.parametrize("k", [2, 5, 16])
def test_many_equal_far_below_the_largest(E, k, score):
    """Logits 16 and more below the largest: equal ones at the border, a larger one at any index."""
    k = min(k, E - 8)
    logits = torch.zeros(70, E, device=DEV)
    logits[:, 5:5 + k - 1] = 20.0 + torch.arange(k - 1, device=DEV)
    logits[:, E - 2] = 1.0
    check(permuted(logits, E), k, score)
    logits[:, E - 2] = 0.0  # all the others equal: the lowest indices
    check(permuted(logits, E + 1), k, score)


@SCORES
@pytest.mark.parametrize("E", SIZES)
def test_masked_by_the_lowest_value(E, score):
    """A finite lowest value as a mask: what is not masked comes first, however far below the largest."""
    for low in (LOWEST, -3e38, -1e4):
        logits = torch.full((67, E), low, device=DEV)
        logits[:, 5] = 2.0
        logits[:, E - 3] = -15.0
        check(permuted(logits, E), 2, score)
        check(permuted(logits, E).bfloat16(), 3, score)


@SCORES
@pytest.mark.parametrize("E", SIZES)
@pytest.mark.parametrize("groups,kept", [(1, 1), (2, 1)])
def test_scores_that_saturate(E, groups, kept, score):
    """Two equal logits and a larger one whose scores are 1 but for 1e-7, a bias of zeros."""
    E = E // groups * groups
    logits = torch.zeros(66, E, device=DEV)
    logits[:, 0] = logits[:, 1] = 16.0
    logits[:, 2 if groups == 1 else E // 2 - 1] = 16.125
    zeros = torch.zeros(E, device=DEV)
    for k in (1, 2):
        check(logits, k, score, zeros, groups, kept)
        check(permuted(logits, E).bfloat16(), k, score, zeros, groups, kept)


@SCORES
@pytest.mark.parametrize("E", SIZES)
@pytest.mark.parametrize("size", [-1e9, 1e9, -1e4])
def test_one_large_bias(E, size, score):
    """One expert's finite bias so large that the others' scores collapse into one value of fp32."""
    logits = randn(E, 400, E).bfloat16()
    bias = torch.zeros(E, device=DEV)
    bias[3] = size
    for k in (1, 4):
        check(logits, k, score, bias)
    if E % 4 == 0:
        check(logits, 3, score, bias, 4, 2)


@SCORES
@pytest.mark.parametrize("E", SIZES)
@pytest.mark.parametrize("biased", [False, True])
def test_few_values(E, biased, score):
    """Rows of few values, near and far apart, in any order: many equal at every border."""
    g = torch.Generator(device=DEV)
    g.manual_seed(E)
    values = torch.tensor([16.0, 16.125, 0.0, 0.0, 0.0, 1.0, -1.0, -40.0, LOWEST, -3e38, 3.0, 3.0000002], device=DEV)
    logits = values[torch.randint(0, len(values), (150, E), generator=g, device=DEV)]
    logits[::3] = torch.where(logits[::3] > 2, 0.0, logits[::3])
    bias = None
    if biased:
        sizes = torch.tensor([0.0, 0.0, 0.0, 0.5, -1e9, 1e6], device=DEV)
        bias = sizes[torch.randint(0, len(sizes), (E,), generator=g, device=DEV)]
    for k in (1, 6):
        check(logits, k, score, bias)
        if E % 8 == 0:
            check(logits, min(k, E // 8 * 3), score, bias, 8, 3)


@SCORES
@pytest.mark.parametrize("E,groups", [(16, 8), (32, 8), (60, 6), (64, 8), (128, 8), (256, 8), (320, 8), (512, 16), (1024, 64)])
def test_groups_whose_sums_overflow(E, groups, score):
    """A group counts the sum of two: with biases of the type's lowest or largest values it passes fp32."""
    per = E // groups
    k = min(16, per + 1)
    for equal in (False, True):
        logits = torch.zeros(66, E, device=DEV) if equal else randn(E, 66, E)
        bias = torch.full((groups, per), LOWEST, device=DEV)
        bias[3] = 0.0  # all groups but one masked, two kept
        check(logits, k, score, bias.flatten(), groups, 2)
        bias[1] = -3e38  # better than the lowest
        check(logits, k, score, bias.flatten(), groups, 2)
        check(logits, k, score, bias.flatten(), groups, 3)
        bias[:] = 0.1
        bias[2], bias[4] = 3e38, 3.3e38
        check(logits, min(per, 16), score, bias.flatten(), groups, 1)
        bias[0, 0], bias[0, 1] = -LOWEST, LOWEST
        check(logits, k, score, bias.flatten(), groups, 2)
        bias[5] = -LOWEST
        check(logits, k, score, bias.flatten(), groups, 3)
