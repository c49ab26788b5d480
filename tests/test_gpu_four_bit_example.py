"""The 4-bit example runs, and what it reports belongs to what it emits."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_rounds(fmt):
    from four_bit_head import FourBitRounds

    r = FourBitRounds(B=3, vocab=1000, dim=128, fmt=fmt)
    for _ in range(3):
        accepted, tokens, logprobs = r.step()
        torch.cuda.synchronize()
        assert ((accepted >= 0) & (accepted <= r.layers)).all()
        emitted = torch.arange(tokens.shape[1], device=tokens.device)[None] <= accepted[:, None]
        assert ((tokens >= 0) == emitted).all()
        assert (torch.isfinite(logprobs) == emitted).all() and (logprobs <= 0).all()
        assert (r.root >= 0).all()
