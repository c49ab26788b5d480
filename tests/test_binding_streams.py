"""Every call with stream=... allocates on that stream, the older ones as the paged ones (the
library and the CUDA side of torch are stand-ins)."""
import pytest
import torch

from speculative_decoding_tree_spec_gb300 import binding
from test_paged_streams import FakeLib, FakeStream, FakeTensor, FakeTorch

I32, F32, BF = torch.int32, torch.float32, torch.bfloat16


class Tensor(FakeTensor):
    def stride(self, i=None):
        return self._strides if i is None else self._strides[i]

    def __getitem__(self, at):  # views: one memory
        return self

    def view(self, *shape):
        return self

    def to(self, *a):
        return self

    def __and__(self, other):
        return self


class Torch(FakeTorch):
    def empty(self, shape, dtype=None, device=None):
        t = super().empty(shape, dtype, device)
        made = Tensor(t.shape, t.dtype, t.dev, t.made_on)
        self.cuda.made[-1] = made
        return made


class Lib(FakeLib):
    def __getattr__(self, name):
        return (lambda *a: 1024) if "workspace_size" in name else super().__getattr__(name)


def T(shape, dtype):
    return Tensor(shape, dtype, 0)


P, IDS = T((2, 3, 64), F32), T((2, 3), I32)
W, X = T((64, 32), BF), T((6, 32), BF)
CALLS = {
    "verify_tree": lambda s: binding.verify_tree(P, P, IDS, IDS, 2, 1.0, stream=s),
    "verify_tree_per_request": lambda s: binding.verify_tree_per_request(
        P, P, IDS, IDS, 2, T((2,), F32), stream=s),
    "verify_tree_fused_lmhead": lambda s: binding.verify_tree_fused_lmhead(
        X, W, None, IDS, IDS, 2, 0.0, stream=s),
    "draft_topk": lambda s: binding.draft_topk(T((6, 64), F32), 4, stream=s),
    "draft_topk, by place": lambda s: binding.draft_topk(T((6, 64), F32), 4, 1.0, s),
    "draft_topk_fused_lmhead": lambda s: binding.draft_topk_fused_lmhead(X, W, 4, stream=s),
    "tree_expand_topk": lambda s: binding.tree_expand_topk(IDS, T((2, 3), F32), 0, 3, 2, s),
    "tree_build": lambda s: binding.tree_build(IDS, IDS, T((2, 3), F32), T((2,), I32), 2, stream=s),
    "filter_rows": lambda s: binding.filter_rows(T((6, 64), F32), 1.0, stream=s),
    "philox_words": lambda s: binding.philox_words(1, 2, T((6,), I32), T((6,), I32), stream=s),
}


@pytest.fixture
def fake(monkeypatch):
    t = Torch()
    t.cuda.current_stream = lambda: FakeStream(0, t.cuda.streams[0])
    monkeypatch.setattr(binding, "torch", t)
    monkeypatch.setattr(binding, "_lib", Lib(t.cuda))
    return t.cuda


@pytest.mark.parametrize("stream", ["none", "current", "side"])
@pytest.mark.parametrize("name", CALLS)
def test_allocations_and_launches_go_to_the_stream(fake, name, stream):
    fake.streams[0] = 11
    s = {"none": None, "current": FakeStream(0, 11), "side": FakeStream(0, 77)}[stream]
    raw = 77 if stream == "side" else 11
    CALLS[name](s)
    assert len(fake.calls) == 1 and fake.calls[0][1:] == (0, raw)
    assert fake.made and all(t.made_on == (0, raw) for t in fake.made)
    assert fake.streams[0] == 11
