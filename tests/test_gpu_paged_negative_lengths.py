"""A negative prefix length counts as 0, for the append and the commit alike."""
import numpy as np
import pytest
import torch

from oracle import paged as oracle
from speculative_decoding_tree_spec_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("prefix", [-1, -3, -2 ** 31])
def test_commit_moves_what_append_stored(prefix):
    g = torch.Generator().manual_seed(1)
    N, d, page = 9, 64, 4
    kv = torch.randn((2, 6, page, 1, d), generator=g).to(DEV)
    k = torch.randn((1, N, 1, d), generator=g).to(DEV)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    table, path, acc = i32([[4, 0, 2]]), i32([[0, 2, 5, 8]]), i32([3])
    before = kv.clone()
    for pre, cache in ((prefix, kv), (0, before)):
        binding.paged_append_rope(None, k, k, cache[0], cache[1], table, i32([pre]))
        binding.commit_accepted_path_paged(cache, table, i32([pre]), path, acc)
    assert torch.equal(kv, before)
    rows = kv[0, table[0].long()].reshape(-1, d)
    assert torch.equal(rows[:4], k[0, [0, 2, 5, 8], 0])


def test_commit_of_mixed_lengths():
    rng = np.random.default_rng(2)
    cache = rng.integers(-30000, 30000, (3, 12, 5, 2, 8)).astype(np.int16)
    table = rng.permutation(12).astype(np.int32).reshape(3, 4)
    prefix = np.array([-4, 6, -1], dtype=np.int32)
    path = np.array([[0, 3, 4, 9], [0, 2, 7, -1], [0, 1, 2, 6]], dtype=np.int32)
    acc = np.array([3, 2, 3], dtype=np.int32)
    want = oracle.commit(cache, table, np.maximum(prefix, 0), path, acc)
    np.testing.assert_array_equal(oracle.commit(cache, table, prefix, path, acc), want)
    t = lambda x: torch.as_tensor(x, device=DEV)
    dev = t(cache)
    binding.commit_accepted_path_paged(dev, t(table), t(prefix), t(path), t(acc))
    np.testing.assert_array_equal(dev.cpu().numpy(), want)
