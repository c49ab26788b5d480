"""Products whose weight rows end inside a tile, on CTAs that take whole tiles and the last one in turn,
with more than one piece of 32 activation rows: exact, every time.  The reference is a product in 64
bits of numbers whose sums fp32 holds, so there is no tolerance but bf16's one rounding, which torch
does on the exact value."""
import pytest
import torch

from oracle import fp4 as oracle_fp4
from speculative_decoding_tree_spec_gb300 import binding
from test_gpu_fp4 import _matrix, _random

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
K = 64


@pytest.fixture(scope="module", params=["mx", "nv"])
def head(request):
    """The format, a weight of 151936 rows and its values."""
    w = _random(151936, K, request.param, 1)
    return request.param, w, torch.from_numpy(oracle_fp4.values(*w, request.param)).to(DEV)


def _check(head, R, V, repeats):
    fmt, (codes, scales), values = head
    a = _random(R, K, fmt, R)
    want = torch.from_numpy(oracle_fp4.values(*a, fmt)).to(DEV) @ values[:V].T
    # products are multiples of 2^-8 (mx: 2^-6), and 24 bits hold their partial sums in any order
    size = torch.from_numpy(abs(oracle_fp4.values(*a, fmt))).to(DEV) @ values[:V].abs().T
    assert size.max() < 2.0 ** -8 * 2 ** 24
    am, wm = _matrix(*a, fmt), _matrix(codes[:V], scales[:V], fmt)
    for dtype in (F32, BF):
        exact = want.to(F32).to(dtype)
        for _ in range(repeats):
            assert torch.equal(binding.fp4_linear(am, wm, dtype), exact)


@pytest.mark.parametrize("R", [64, 200, 640])
@pytest.mark.parametrize("V", [151936, 50257])
def test_vocabularies_that_end_inside_a_tile(head, V, R):
    _check(head, R, V, 20)


@pytest.mark.parametrize("R", [60, 192, 700])
@pytest.mark.parametrize("V", [128 * 156 + 1, 128 * 156 + 33, 128 * 457 + 97])
def test_last_tiles_of_one_to_four_warps(head, V, R):
    """1, 33 and 97 rows in the last tile: warps with no row, with some and with all in one tile."""
    _check(head, R, V, 20)
