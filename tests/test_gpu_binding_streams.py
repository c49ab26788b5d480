"""verify_tree and its end-to-end call on a side stream, outputs and workspaces the call's own."""
import pytest
import torch

from speculative_decoding_tree_spec_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _tensors(seed, pinned=False):
    g = torch.Generator().manual_seed(seed)
    B, N, V = 8, 15, 4096
    p, q = (torch.randn((B, N, V), generator=g).to(torch.bfloat16) for _ in range(2))
    tok = torch.randint(0, V, (B, N), generator=g, dtype=torch.int32)
    par = torch.tensor([-1] + [(n - 1) // 2 for n in range(1, N)], dtype=torch.int32).repeat(B, 1)
    return [x.pin_memory() if pinned else x.to(DEV) for x in (p, q, tok, par)]


def test_two_side_streams_at_once():
    data = [_tensors(s) for s in (1, 2)]
    want = [binding.verify_tree(*d, 3, 1.0, seed=5) for d in data]
    side = [torch.cuda.Stream() for _ in data]
    torch.cuda.synchronize()
    for _ in range(50):
        got = [binding.verify_tree(*d, 3, 1.0, seed=5, stream=s) for d, s in zip(data, side)]
        torch.full((1 << 23,), float("nan"), device=DEV)
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            for k in ("accept_len", "tokens", "path", "status"):
                assert torch.equal(g[k], w[k]), k
            # bits: alpha is NaN at the nodes that the walk does not reach
            assert torch.equal(g["alpha"].view(torch.int32), w["alpha"].view(torch.int32))


def test_host_call_and_counters_on_a_side_stream():
    host = _tensors(3, pinned=True)
    want = binding.verify_tree_host(*host, 3, 1.0, seed=5)
    for _ in range(20):
        got = binding.verify_tree_host(*host, 3, 1.0, seed=5, stream=torch.cuda.Stream())
        for k in ("accept_len", "tokens", "path"):
            assert torch.equal(got[k], want[k])
    d = _tensors(3)
    a = binding.PreparedVerify(*d, 3, 1.0, seed=5).read_counters()
    b = binding.PreparedVerify(*d, 3, 1.0, seed=5, stream=torch.cuda.Stream()).read_counters()
    assert a == b
    x = binding.verify_tree(*d, 3, 1.0, seed=5, want_counters=True, stream=torch.cuda.Stream())
    assert x["counters"]["dense_rows"] == a["dense_rows"]
