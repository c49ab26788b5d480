"""Calls handed to side streams (stream=...) from the default stream, without workspaces and
outputs of the caller's."""
import numpy as np
import pytest
import torch

from speculative_decoding_tree_spec_gb300 import binding
from test_gpu_paged import BF, DEV, F32, Case

pytestmark = pytest.mark.gpu


class RoomyCase(Case):
    room = 5000  # no clusters: parts of tiles go through the workspace


def _args(c):
    return ([c.device(x) for x in (c.q, c.k, c.v, c.table, c.prefix)] + [c.scale],
            dict(mask=c.device(c.mask), shared_len=c.shared))


@pytest.mark.parametrize("dtype,N,shared", [(BF, 40, 0), (BF, 40, 160), (BF, 2, 0), (F32, 6, 0)])
def test_two_streams_at_once(dtype, N, shared):
    cases = [RoomyCase([shared + 3000, shared + 50 * b, shared + 900], N, 8, 2, 128, 16, dtype, seed=b,
                       mask="tree", shared=shared) for b in (1, 2)]
    dev = [_args(c) for c in cases]
    want = [binding.tree_attention_paged(*a, **kw) for a, kw in dev]
    side = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(60):
        got = []
        for s, (a, kw) in zip(side, dev):
            for _ in range(2):
                last = binding.tree_attention_paged(*a, **kw, stream=s)
            got.append(last)
            # the next owner of memory that belongs to the default stream
            torch.full((1 << 24,), float("nan"), device=DEV)
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g["out"], w["out"]) and torch.equal(g["lse"], w["lse"])
    cases[0].check(want[0])


def test_a_round_on_a_side_stream():
    """Append, attention and commit with stream=..., the queries allocated by the call."""
    c = RoomyCase([70, 3], 9, 4, 2, 64, 16, seed=1, mask="tree", pad_nan=False)
    k = torch.randn((2, 9, 2, 64), generator=torch.Generator().manual_seed(2)).to(BF).to(DEV)
    t = lambda x: torch.as_tensor(np.asarray(x, dtype=np.int32), device=DEV)
    q, table, pre, mask = c.device(c.q), c.device(c.table), c.device(c.prefix), c.device(c.mask)
    path, acc = t([[0, 2, 5, 8], [0, 1, 4, 6]]), t([3, 2])
    ang = torch.arange(100, device=DEV)[:, None] * 0.1 ** torch.arange(32, device=DEV)
    cs = torch.cat([ang.cos(), ang.sin()], dim=1).float()
    results = []
    side = torch.cuda.Stream()
    for s in (None, side):
        cache = torch.stack([c.device(c.k), c.device(c.v)])
        torch.cuda.synchronize()
        rq = binding.paged_append_rope(q, k, k, cache[0], cache[1], table, pre, cs, stream=s)
        out = binding.tree_attention_paged(rq, cache[0], cache[1], table, pre, mask=mask, stream=s)
        binding.commit_accepted_path_paged(cache, table, pre, path, acc, stream=s)
        torch.cuda.synchronize()
        results.append((rq, out["out"], out["lse"], cache))
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_an_external_stream_and_a_captured_side_stream():
    c = RoomyCase([300, 20], 20, 8, 2, 64, 16, seed=3, mask="tree")
    a, kw = _args(c)
    want = binding.tree_attention_paged(*a, **kw)
    s = torch.cuda.Stream()
    ext = torch.cuda.ExternalStream(s.cuda_stream)
    torch.cuda.synchronize()
    got = binding.tree_attention_paged(*a, **kw, stream=ext)
    torch.cuda.synchronize()
    assert torch.equal(got["out"], want["out"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.wait_stream(torch.cuda.current_stream())
        got = binding.tree_attention_paged(*a, **kw, stream=s)
        torch.cuda.current_stream().wait_stream(s)
    for _ in range(3):
        got["out"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])
