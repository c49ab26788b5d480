"""The decoding rounds of examples/paged_round.py: what a round leaves in the paged cache is
what caching the accepted sequence from its start would have left."""
import os
import sys

import numpy as np
import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))
from paged_round import PagedRounds  # noqa: E402

pytestmark = pytest.mark.gpu


def _rows(r, b, n):
    t = np.arange(n)
    pages = r.table[b].cpu().numpy()[t // r.page_size].astype(np.int64)
    at = torch.as_tensor(pages, device=r.device), torch.as_tensor(t % r.page_size, device=r.device)
    return r.cache[:, at[0], at[1]]


def test_rounds_leave_the_cache_of_the_accepted_sequence():
    r = PagedRounds(seed=3)
    counts = torch.tensor([40, 1, 17, 33], dtype=torch.int32, device=r.device)
    prompt = torch.randint(0, r.vocab, (r.B, 40), dtype=torch.int32, device=r.device,
                           generator=torch.Generator(device=r.device).manual_seed(2))
    r.prefill(prompt, counts)
    seqs = [prompt[b, :int(counts[b])].tolist() for b in range(r.B)]
    moved = 0
    for _ in range(6):
        accepted, tokens = r.step()
        for b, (a, t) in enumerate(zip(accepted.tolist(), tokens.tolist())):
            assert a >= 0
            moved += a
            seqs[b] += t[:a + 1]
    assert moved > 0  # the rounds did move accepted rows
    # all but each sequence's last token are cached; the same tokens cached at once, in order
    fresh = PagedRounds(seed=3)
    longest = max(len(s) for s in seqs) - 1
    tokens = torch.tensor([(s + [0] * longest)[:longest] for s in seqs], dtype=torch.int32,
                          device=r.device)
    n = torch.tensor([len(s) - 1 for s in seqs], dtype=torch.int32, device=r.device)
    assert torch.equal(n, r.length)
    fresh.attend(tokens, counts=n)
    for b in range(r.B):
        # one projection is a library product whose tiling may go by the batch: a rounding
        got, want = _rows(r, b, len(seqs[b]) - 1).float(), _rows(fresh, b, len(seqs[b]) - 1).float()
        assert (got - want).abs().max() <= 2 ** -7 * want.abs().max()
