"""A negative prefix length counts as 0 in every paged operator's oracle."""
import numpy as np

from oracle import paged


def test_commit_follows_the_append():
    rng = np.random.default_rng(0)
    N, page = 8, 3
    x = rng.standard_normal((1, N, 1, 4))
    table = np.array([[2, 0, 3]])
    path, acc = np.array([[0, 2, 4, 7]]), np.array([3])
    left = []
    for prefix in (0, -1, -6):
        cache = np.zeros((4, page, 1, 4))
        _, kc, _ = paged.append(x, x, x, cache, cache, table, np.array([prefix]), np.zeros((1, 0)))
        left.append(paged.commit(kc[None], table, np.array([prefix]), path, acc)[0])
    rows = left[0][table[0]].reshape(-1, 4)
    np.testing.assert_array_equal(rows[:4], x[0, [0, 2, 4, 7], 0])
    np.testing.assert_array_equal(left[1], left[0])
    np.testing.assert_array_equal(left[2], left[0])
