"""Row numbers by the hundred: none, some and all of them without a row, in any order.  Tolerances:
tests/test_gpu_logprobs.py."""
import numpy as np
import pytest
import torch

from speculative_decoding_tree_spec_gb300 import binding
from test_gpu_logprobs import BF, DEV, _check, _gauss

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("missing", [0.0, 0.5, 1.0])
@pytest.mark.parametrize("R", [152, 305, 448, 457, 700])
def test_row_numbers_by_the_hundred(R, missing):
    g = np.random.default_rng(R)
    n, V = 300, 5001
    rows = np.where(g.random(R) < missing, g.choice([-1, n, 2 ** 31 - 1], R), g.integers(0, n, R))
    x = _gauss(n, V, R)
    got = _check(x, BF, g.integers(0, V, (R, 2)), 5, 0.9, rows)
    assert (got["status"].cpu().numpy() == np.where((rows >= 0) & (rows < n), 0, 4)).all()


@pytest.mark.parametrize("R", [305, 448])
def test_a_permutation_gives_the_rows(R):
    """The rows by their numbers in any order and the rows laid out in that order: bit for bit the same."""
    V = 128256
    x = torch.randn((R, V), generator=torch.Generator(device=DEV).manual_seed(R), device=DEV).to(BF)
    order = torch.randperm(R, generator=torch.Generator().manual_seed(1)).to(DEV)
    tokens = torch.randint(0, V, (R,), device=DEV, dtype=torch.int32)
    got = binding.token_logprobs(x, tokens, 5, rows=order.to(torch.int32))
    want = binding.token_logprobs(x[order].contiguous(), tokens, 5)
    assert all(torch.equal(got[k], want[k]) for k in want)
