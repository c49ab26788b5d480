"""The oracle of the paged-cache operators against results worked out another way."""
import numpy as np

from oracle import commit as oracle_commit
from oracle import paged


def test_slot_pages_and_holes():
    table = [4, -1, 0, 9]
    assert paged.slot(table, 5, 3, 2) == (4, 2)
    assert paged.slot(table, 5, 3, 7) == (0, 1)
    for t in (-1, 3, 9, 12):  # before the start, no page, beyond the cache, beyond the table
        assert paged.slot(table, 5, 3, t) is None


def test_rotation_by_a_quarter_turn_and_its_inverse():
    x = np.array([1.0, 2.0, 3.0, 4.0, 5.0])
    quarter = np.array([0.0, 0.0, 1.0, 1.0])  # cos 0, sin 1
    np.testing.assert_array_equal(paged.rotate(x, quarter, False), [-3, -4, 1, 2, 5])
    np.testing.assert_array_equal(paged.rotate(x, quarter, True), [-2, 1, -4, 3, 5])
    a = np.array([0.3, 1.1])
    row, back = np.concatenate([np.cos(a), np.sin(a)]), np.concatenate([np.cos(a), -np.sin(a)])
    for inter in (False, True):
        np.testing.assert_allclose(paged.rotate(paged.rotate(x, row, inter), back, inter), x,
                                   rtol=1e-15)


def test_rotated_products_depend_on_the_distance_alone():
    rng = np.random.default_rng(0)
    q, k = rng.normal(size=(2, 8))
    f = 10.0 ** -np.arange(4)
    rows = [np.concatenate([np.cos(p * f), np.sin(p * f)]) for p in range(40)]
    for inter in (False, True):
        dots = [paged.rotate(q, rows[p + 5], inter) @ paged.rotate(k, rows[p], inter)
                for p in (0, 3, 34)]
        np.testing.assert_allclose(dots, dots[0], rtol=1e-12)


def test_append_stores_where_the_table_says():
    q = np.ones((2, 2, 1, 2))
    k = np.arange(8.0).reshape(2, 2, 1, 2) + 1
    cache = np.zeros((3, 2, 1, 2))
    table = np.array([[2, 0], [1, -1]])
    _, kc, vc = paged.append(q, k, -k, cache, cache, table, [1, 1], np.zeros((9, 0)))
    # sequence 0: positions 1, 2 -> page 2 slot 1, page 0 slot 0; sequence 1: position 2 has no page
    want = np.zeros_like(cache)
    want[2, 1, 0], want[0, 0, 0], want[1, 1, 0] = k[0, 0, 0], k[0, 1, 0], k[1, 0, 0]
    np.testing.assert_array_equal(kc, want)
    np.testing.assert_array_equal(vc, -want)


def _one(prefix, mask=None, counts=None, shared=0, page=4, seed=1):
    rng = np.random.default_rng(seed)
    B, N, Hq, Hkv, D = 2, 3, 2, 1, 4
    q = rng.normal(size=(B, N, Hq, D))
    pool = rng.normal(size=(8, page, Hkv, D)), rng.normal(size=(8, page, Hkv, D))
    table = np.array([[3, 1, 6, 0], [3, 5, 2, 7]])
    return q, pool, table, paged.attention(q, *pool, table, prefix, 0.5, mask, counts, shared)


def test_attention_is_the_softmax_average_of_the_causal_keys():
    q, (kc, vc), table, (out, lse, _, _) = _one([5, 0])
    for b, pre in enumerate([5, 0]):
        t = np.arange(pre + 3)
        k, v = (c[table[b][t // 4], t % 4, 0] for c in (kc, vc))
        for n in range(3):
            e = np.exp(0.5 * q[b, n] @ k[:pre + n + 1].T)
            np.testing.assert_allclose(out[b, n], e @ v[:pre + n + 1] / e.sum(1, keepdims=True))
            np.testing.assert_allclose(lse[b, n], np.log(e.sum(1)))


def test_attention_rows_that_see_nothing():
    mask = np.zeros((2, 3, 3), dtype=np.uint8)
    _, _, _, (out, lse, _, _) = _one([0, 0], mask)
    assert (out == 0).all() and (lse == -np.inf).all()
    _, _, _, (out, lse, _, _) = _one([5, 5], counts=[2, 0])
    assert (lse[0, :2] > -np.inf).all() and (lse[0, 2] == -np.inf).all() and (out[1] == 0).all()


def test_shared_positions_are_an_ordinary_prefix():
    with_, without = _one([6, 5], shared=4)[3], _one([6, 5])[3]
    np.testing.assert_array_equal(with_[0], without[0])
    _, _, _, (out, lse, _, _) = _one([6, 3], shared=4)  # 3 < 4: not behind the shared positions
    assert (out[1] == 0).all() and (lse[1] == -np.inf).all() and (out[0] != 0).all()


def test_commit_equals_the_contiguous_commit_through_the_table():
    rng = np.random.default_rng(3)
    P, B, page, H, R = 2, 3, 4, 2, 5
    table = rng.permutation(12).reshape(B, 4).astype(np.int32)
    cache = rng.integers(0, 255, (P, 12, page, H, R)).astype(np.uint8)
    prefix, path, acc = [3, 9, 0], [[0, 2, 5], [0, 1, 6], [0, 4, -1]], [2, 2, -1]
    flat = cache[:, table].reshape(P, B, 16, H * R)
    want = oracle_commit.commit_accepted_path(flat, prefix, path, acc)
    got = paged.commit(cache, table, prefix, path, acc)
    np.testing.assert_array_equal(got[:, table].reshape(P, B, 16, H * R), want)
