"""Causal attention (no mask) over page tables with holes: only the positions of a page that
the table lacks are masked, whatever blocks are looked at together with them.  Tolerances:
tests/test_gpu_paged.py."""
import pytest
import torch

from test_gpu_paged import BF, Case

pytestmark = pytest.mark.gpu


class RoomyCase(Case):
    room = 5000  # many rows then go to the tensor-memory kernel


def _holes(prefix, N):
    """Page entries: in the prefix or at the start, among the drafts, near the end, and just behind
    what the sequence holds."""
    last = (prefix + N - 1) // 16
    return sorted({0, 2, min(prefix // 16 + 1, last), last, last + 1})


@pytest.mark.parametrize("dtype", [BF, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("prefix", [0, 127, 130])
@pytest.mark.parametrize("N", [20, 64, 600])
def test_holes_mask_their_own_positions_alone(prefix, N, dtype):
    if dtype is not BF and N > 64:
        pytest.skip("the few-rows kernel has no case of its own there")
    for hole in _holes(prefix, N):
        c = RoomyCase([prefix, 5], N, 8, 2, 64, 16, dtype, seed=N + hole)
        c.table[0, hole] = -1
        c.check()


@pytest.mark.parametrize("hq,hkv", [(8, 2), (2, 2), (6, 2)])
def test_holes_in_several_blocks_and_padding(hq, hkv):
    N = 300
    c = RoomyCase([90, 0, 257], N, hq, hkv, 64, 16, seed=hq, counts=[N, 270, 131])
    c.table[0, [3, 20]] = 1 << 20
    c.table[1, [1, 9]] = -1
    c.table[2, 17] = c.k.shape[0]
    c.check()
