"""Pins of the log-probability oracle: closed forms, brute-force ranks, the entropy's bounds and identities."""
import math

import numpy as np

from oracle.logprobs import token_logprobs


def test_two_levels_in_closed_form():
    V, a, b, T = 100, 2.0, -1.0, 0.8
    z = np.full((1, V), b, dtype=np.float32)
    z[0, 37] = a
    r = token_logprobs(z, [[37, 0]], 3, T)
    e = math.exp((b - a) / T)
    s = 1 + (V - 1) * e
    assert abs(r["logprobs"][0, 0] + math.log(s)) < 1e-12
    assert abs(r["logprobs"][0, 1] - ((b - a) / T - math.log(s))) < 1e-12
    p = np.array([1 / s] + [e / s] * (V - 1))
    assert abs(r["entropy"][0] + (p * np.log(p)).sum()) < 1e-12
    assert r["top_tokens"][0].tolist() == [37, 0, 1]


def test_uniform_and_certain_rows():
    r = token_logprobs(np.zeros((1, 64), dtype=np.float32), [[5]], 2)
    assert abs(r["entropy"][0] - math.log(64)) < 1e-12 and abs(r["logprobs"][0, 0] + math.log(64)) < 1e-12
    z = np.full((1, 9), -np.inf, dtype=np.float32)
    z[0, 4] = 3.0
    r = token_logprobs(z, [[4, 0]], 2)
    assert r["entropy"][0] == 0 and r["logprobs"][0].tolist() == [0, -np.inf]
    assert r["top_tokens"][0].tolist() == [4, 0] and r["top_logprobs"][0].tolist() == [0, -np.inf]


def test_ranks_by_counting():
    rng = np.random.default_rng(1)
    for _ in range(30):
        V = int(rng.integers(2, 40))
        z = (rng.integers(-4, 5, size=(1, V)) * 0.5).astype(np.float32)
        r = token_logprobs(z, None, V)
        for rank, t in enumerate(r["top_tokens"][0]):
            assert rank == sum(z[0, j] > z[0, t] or (z[0, j] == z[0, t] and j < t) for j in range(V))
        assert abs(np.exp(r["top_logprobs"]).sum() - 1) < 1e-12
        assert abs(r["entropy"][0] + (np.exp(r["top_logprobs"]) * r["top_logprobs"]).sum()) < 1e-12


def test_small_probabilities_keep_their_digits():
    z = np.zeros((1, 11), dtype=np.float32)
    z[0, 0] = 50.0
    r = token_logprobs(z, [[0]], 0)
    assert abs(r["logprobs"][0, 0] / -(10 * math.exp(-50)) - 1) < 1e-12


def test_rows_tokens_and_status():
    z = np.array([[0, 1], [np.nan, 0], [np.inf, 0], [-np.inf, -np.inf], [2, -np.inf]], dtype=np.float32)
    r = token_logprobs(z, [[0], [0], [0], [0], [2], [-1], [0]], 1, 1.0, [0, 1, 2, 3, 4, 0, 5])
    assert r["status"].tolist() == [0, 1, 1, 1, 0, 0, 4]
    assert np.isnan(r["logprobs"][1:4]).all() and np.isneginf(r["logprobs"][4:7]).all()
    assert r["top_tokens"][:, 0].tolist() == [1, -1, -1, -1, 0, 1, -1]
    bits = (np.array([[1.5, -2.0]], dtype=np.float32).view(np.uint32) >> 16).astype(np.uint16)
    a, b = token_logprobs(bits, [[0]]), token_logprobs(np.array([[1.5, -2.0]], dtype=np.float32), [[0]])
    assert a["logprobs"] == b["logprobs"]
