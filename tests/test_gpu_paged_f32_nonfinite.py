"""Infinities and NaN in fp32 caches and queries: what the formula gives for them must not
depend on how a product is split.  Tolerances: tests/test_gpu_paged.py."""
import numpy as np
import pytest
import torch

from test_gpu_paged import F32, Case, _np

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(autouse=True, params=[0, 5000], ids=["tight", "roomy"])
def _room(request, monkeypatch):
    monkeypatch.setattr(Case, "room", request.param)


def _at(c, b, t, page=16):
    return int(c.table[b, t // page]), t % page


@pytest.mark.parametrize("N", [1, 40])
@pytest.mark.parametrize("d", [64, 128])
def test_infinite_values_reach_everyone_who_sees_them(N, d):
    """Whole pages, so that the keys of weight 1 in their step are among them."""
    c = Case([200, 20, 75], N, 4, 2, d, 16, F32, seed=4, mask="tree")
    c.v[int(c.table[0, 1]), :, 0, 7] = INF
    c.v[int(c.table[0, 6]), :, 1, 8] = -INF
    c.v[int(c.table[1, 0]), 3, 1, 9] = float("nan")
    c.v[_at(c, 2, 70)][0, 3] = INF
    c.v[_at(c, 2, 9)][0, 3] = -INF  # with the one above: NaN
    got = c.check()
    assert torch.isposinf(got["out"][0, :, :2, 7]).all()
    assert torch.isneginf(got["out"][0, :, 2:, 8]).all()
    assert torch.isnan(got["out"][2, :, :2, 3]).all()


def test_an_infinite_value_of_the_only_visible_key():
    c = Case([1], 1, 2, 1, 64, 16, F32, mask=np.zeros((1, 1, 1), dtype=np.uint8))
    c.v[_at(c, 0, 0)][0, 5] = INF
    got = c.check()
    assert torch.isposinf(got["out"][0, 0, :, 5]).all()


def test_infinite_values_of_shared_positions_and_of_long_contexts():
    c = Case([160, 170, 190], 3, 4, 2, 64, 16, F32, mask="tree", shared=160)
    c.v[int(c.table[0, 2]), :, 0, 7] = INF
    c.v[int(c.table[2, 10]), :10, 1, 3] = -INF
    c.check()
    c = Case([9000], 2, 2, 1, 64, 16, F32, seed=1)
    c.v[int(c.table[0, 300]), :, 0, 11] = INF
    c.check()


@pytest.mark.parametrize("N", [1, 9])
def test_a_key_that_scores_minus_infinity_has_no_weight(N):
    """-inf against query elements that are exact in few bits: as if the key were not there."""
    c = Case([40, 77], N, 4, 2, 64, 1, F32, seed=N)
    c.q[..., 3] = 1.0
    places = [(0, 7), (0, 39), (1, 0), (1, 64)]
    for b, t in places:
        c.k[int(c.table[b, t]), 0, :, 3] = -INF
    got = c.run()
    for b, t in places:
        c.table[b, t] = -1
    c.check(got)


def test_infinite_queries():
    """+inf or -inf scores: NaN where the formula's inf - inf is, one key's value where all other
    scores are -inf."""
    c = Case([30], 1, 2, 1, 64, 1, F32, seed=3)
    c.q[0, 0, :, 2] = -INF
    c.k[..., 2] = 1.0           # every score -inf ...
    c.k[int(c.table[0, 12]), 0, 0, 2] = -1.0  # ... but this one: inf
    got = c.run()
    assert torch.isnan(got["out"]).all()
    c.q[0, 0, :, 2] = 1.0
    c.k[..., 2] = -INF
    c.k[int(c.table[0, 12]), 0, 0, 2] = -1.0
    got = c.run()
    want = c.v[int(c.table[0, 12]), 0, 0]
    err = (got["out"][0, 0].cpu() - want).abs()
    assert (err <= 2.0 ** -20 * want.abs()).all()  # one value through split products, weight 1


def test_nan_with_a_payload_in_the_low_bits_stays_nan():
    low = torch.tensor([0x7F800001], dtype=torch.int32).view(torch.float32)
    c = Case([60, 33], 5, 4, 2, 64, 16, F32, seed=5)
    c.v[_at(c, 0, 17)][1, 6:7] = low
    c.k[_at(c, 1, 20)][0, 9:10] = low
    got = c.check()
    assert torch.isnan(got["out"][0, :, 2:, 6]).all()
    assert torch.isnan(got["out"][1, :, :2]).all() and torch.isfinite(got["out"][1, :, 2:]).all()
    assert np.isnan(_np(got["lse"])[1, :, :2]).all()
