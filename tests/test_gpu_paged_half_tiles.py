"""Tiles of one and of two halves in turn within a CTA, all with drafts whose values are not
finite among them.  Tolerances: tests/test_gpu_paged.py."""
import numpy as np
import pytest

from test_gpu_paged import Case

pytestmark = pytest.mark.gpu


class RoomyCase(Case):
    room = 5000


@pytest.mark.parametrize("N,hq,hkv", [(75, 8, 2), (300, 1, 1)])  # tiles of 256 and 44 rows
@pytest.mark.parametrize("mask", ["tree", None], ids=["tree", "causal"])
def test_tiles_of_one_and_two_halves_in_turn(N, hq, hkv, mask):
    B = 100 * 2 // hkv
    c = RoomyCase([7 * b % 41 for b in range(B)], N, hq, hkv, 64, 16, seed=N, mask=mask)
    for b in range(0, B, 9):
        t = int(c.prefix[b]) + 5 + b % 20
        c.v[int(c.table[b, t // 16]), t % 16][0, b % 64] = np.inf
    c.check()
