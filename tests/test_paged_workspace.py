"""A workspace handed to tree_attention_paged: only one contiguous tensor on the cache's device,
counted in bytes (the library and the CUDA side of torch are stand-ins)."""
import pytest
import torch

from speculative_decoding_tree_spec_gb300 import binding
from test_paged_streams import FakeLib, FakeTensor, FakeTorch


@pytest.fixture
def attend(monkeypatch):
    t, calls = FakeTorch(), []
    L = FakeLib(t.cuda)
    L.spec_tree_attention_paged = lambda *a: calls.append(a) or 0
    monkeypatch.setattr(binding, "torch", t)
    monkeypatch.setattr(binding, "_lib", L)
    q, cache = FakeTensor((2, 3, 4, 64), torch.bfloat16, 0), FakeTensor((5, 16, 2, 64), torch.bfloat16, 0)
    table, pre = FakeTensor((2, 2), torch.int32, 0), FakeTensor((2,), torch.int32, 0)
    return (lambda ws: binding.tree_attention_paged(q, cache, cache, table, pre, workspace=ws)), calls


class Strided(FakeTensor):
    def is_contiguous(self):
        return False


@pytest.mark.parametrize("bad", [FakeTensor((4096,), torch.uint8, -1), FakeTensor((4096,), torch.uint8, 1),
                                 Strided((4096,), torch.uint8, 0)], ids=["host", "other device", "strided"])
def test_unusable_workspaces_are_refused(attend, bad):
    call, calls = attend
    with pytest.raises(TypeError):
        call(bad)
    assert not calls


def test_the_size_is_in_bytes(attend):
    call, calls = attend
    call(FakeTensor((700,), torch.bfloat16, 0))  # element_size 2
    assert calls[0][-2] == 1400
