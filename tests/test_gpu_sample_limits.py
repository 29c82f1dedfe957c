"""Sampling where a filter meets a limit of the temperature: tokens equal to those of 64-bit arithmetic."""
import math

import numpy as np
import pytest
import torch

from tests.test_gpu_sample import TYPES, check, logits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("min_p", [1.0, 1.0 - 2.0 ** -24, 0.5, 1e-30])
def test_min_p_where_every_weight_is_1(dtype, min_p):
    """Under an infinite temperature every finite logit has the weight 1, which no min_p up to 1 takes away."""
    rng = np.random.default_rng(21)
    x = logits(9, 4000, dtype, rng)
    x[:, 100:300] = -math.inf
    u, t, m = rng.random(9), [math.inf] * 9, [min_p] * 9
    check(x, t, u, m=m)
    check(x, t, u, k=[70] * 9, m=m)
    check(x, t, u, p=[0.3] * 9, m=m)
    check(x, t, u, k=[700] * 9, p=[0.6] * 9, m=m)
    x[2, 17] = x[2, 3000] = math.inf                             # these share the weight alone
    check(x, t, u, m=m)


def test_min_p_above_1_keeps_the_first_token():
    rng = np.random.default_rng(22)
    x = logits(5, 4000, torch.float32, rng)
    x[:, 3999] = x[:, 7] = x.amax(1)
    for t in (0.8, math.inf):
        check(x, [t] * 5, rng.random(5), m=[1.5] * 5)
