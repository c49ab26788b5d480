"""Logits so far apart that fp32 does not hold their difference, at temperatures for which the quotient
is an ordinary number.  Tolerances: tests/test_gpu_logprobs.py."""
import numpy as np
import pytest
import torch

from test_gpu_logprobs import BF, F32, _check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [4.0, 1e30, 3e37, 2e38, 3.4e38])
@pytest.mark.parametrize("V", [20, 700, 5000, 70001])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_differences_beyond_fp32(dtype, V, T):
    g = np.random.default_rng(V)
    x = torch.from_numpy(g.uniform(-3.3e38, 3.3e38, (6, V)))
    x[0] = torch.linspace(-3.3e38, 3.3e38, V)  # the maximum grows along the row
    x[1] = -x[0]
    x[2, :V // 2] = torch.finfo(dtype).min
    x[2, V // 2] = torch.finfo(dtype).max
    x[3] = float("-inf")
    x[3, 3], x[3, V - 1] = torch.finfo(dtype).min, torch.finfo(dtype).max
    x[4] = torch.finfo(dtype).min
    _check(x, dtype, g.integers(0, V, (6, 3)), 7, T)
