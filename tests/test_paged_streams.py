"""The paged calls' allocations and launches belong to the stream and device they are asked for
(the library and the CUDA side of torch are stand-ins: what is looked at is the binding)."""
import contextlib

import pytest
import torch

from speculative_decoding_tree_spec_gb300 import binding


class FakeStream:
    def __init__(self, device_index, cuda_stream):
        self.device_index, self.cuda_stream = device_index, cuda_stream


class FakeTensor:
    def __init__(self, shape, dtype, dev, made_on=None, strides=None):
        self.shape, self.dtype, self.dev, self.made_on = torch.Size(shape), dtype, dev, made_on
        self.device = torch.device("cuda", dev) if dev >= 0 else torch.device("cpu")
        self._strides = tuple(torch.empty(shape, device="meta").stride()) if strides is None else strides

    def stride(self):
        return self._strides

    def get_device(self):
        return self.dev

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return id(self)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return 2

    def dim(self):
        return len(self.shape)


class Cuda:
    """Current device and each device's current stream, as torch keeps them."""
    Stream = FakeStream

    def __init__(self):
        self.current, self.streams, self.made, self.calls = 0, {0: 0, 1: 0}, [], []

    @contextlib.contextmanager
    def device(self, dev):
        before, self.current = self.current, dev
        yield
        self.current = before

    @contextlib.contextmanager
    def stream(self, s):
        with self.device(s.device_index):
            before, self.streams[s.device_index] = self.streams[s.device_index], s.cuda_stream
            yield
            self.streams[s.device_index] = before

    def default_stream(self, dev):
        return FakeStream(dev, 0)

    def ExternalStream(self, raw, device):
        assert raw  # torch takes 0 for a new stream
        return FakeStream(device, raw)


class FakeTorch:
    def __init__(self):
        self.cuda = Cuda()
        self._C = self

    def __getattr__(self, name):
        return getattr(torch, name)

    def _cuda_getDevice(self):
        return self.cuda.current

    def _cuda_getCurrentRawStream(self, dev):
        return self.cuda.streams[dev]

    def empty(self, shape, dtype=None, device=None):
        shape = (shape,) if isinstance(shape, int) else shape
        dev = torch.device(device).index
        t = FakeTensor(shape, dtype, dev, made_on=(dev, self.cuda.streams[dev]))
        self.cuda.made.append(t)
        return t


class FakeLib:
    def __init__(self, cuda):
        self.cuda = cuda

    def spec_tree_attention_workspace_size(self, *a):
        return 1024

    def __getattr__(self, name):
        def call(*a):
            self.cuda.calls.append((name, self.cuda.current, a[-1]))
            return 0
        return call


@pytest.fixture
def fake(monkeypatch):
    t = FakeTorch()
    monkeypatch.setattr(binding, "torch", t)
    monkeypatch.setattr(binding, "_lib", FakeLib(t.cuda))
    return t.cuda


def _calls(dev):
    bf, i32 = torch.bfloat16, torch.int32
    q, k = FakeTensor((2, 3, 4, 64), bf, dev), FakeTensor((2, 3, 2, 64), bf, dev)
    cache = FakeTensor((5, 16, 2, 64), bf, dev)
    both = FakeTensor((2, 5, 16, 2, 64), bf, dev)
    table, pre, path = (FakeTensor(s, i32, dev) for s in ((2, 2), (2,), (2, 3)))
    return [lambda s: binding.paged_append_rope(q, k, k, cache, cache, table, pre, stream=s),
            lambda s: binding.tree_attention_paged(q, cache, cache, table, pre, stream=s),
            lambda s: binding.commit_accepted_path_paged(both, table, pre, path, pre, stream=s)]


class OtherStream:  # not one of torch's
    cuda_stream = 88


class DefaultStream:
    cuda_stream = 0


@pytest.mark.parametrize("dev", [0, 1])
@pytest.mark.parametrize("stream", ["none", "current", "side", "other", "default"])
@pytest.mark.parametrize("call", [0, 1, 2], ids=["append", "attend", "commit"])
def test_allocations_and_launches_go_to_the_stream(fake, dev, stream, call):
    fake.streams[dev] = 11
    s = {"none": None, "current": FakeStream(dev, 11), "side": FakeStream(dev, 77),
         "other": OtherStream(), "default": DefaultStream()}[stream]
    raw = {"none": 11, "current": 11, "side": 77, "other": 88, "default": 0}[stream]
    _calls(dev)[call](s)
    assert len(fake.calls) == 1 and fake.calls[0][1:] == (dev, raw)  # current device, stream
    assert len(fake.made) == (1, 3, 0)[call]
    assert all(t.made_on == (dev, raw) for t in fake.made)
    assert fake.current == 0 and fake.streams[dev] == 11  # as they were


@pytest.mark.parametrize("call", [0, 1, 2], ids=["append", "attend", "commit"])
def test_a_stream_of_another_device_is_refused(fake, call):
    with pytest.raises(ValueError):
        _calls(0)[call](FakeStream(1, 77))
    assert not fake.calls and not fake.made
