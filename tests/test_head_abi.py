"""The 4-bit and log-probability entry points refuse bad arguments on the host, before anything is
launched (the calls run in a child process that sees no GPU: tests/head_validation_cases.py), and the
binding refuses what does not fit together."""
import json
import os
import subprocess
import sys

import pytest
import torch

import __graft_entry__
import head_validation_cases as hv
from speculative_decoding_tree_spec_gb300 import binding
from test_paged_streams import FakeLib, FakeTensor, FakeTorch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


@pytest.fixture(scope="module")
def codes():
    __graft_entry__.build()
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    env["PYTHONPATH"] = os.pathsep.join([ROOT, here, env.get("PYTHONPATH", "")])
    r = subprocess.run([sys.executable, os.path.join(here, "head_validation_cases.py")], capture_output=True,
                       text=True, env=env, cwd=ROOT, timeout=300)
    assert r.returncode == 0, r.stderr
    return json.loads(r.stdout)


@pytest.mark.parametrize("name,cases", [("quantize", hv.QUANTIZE), ("dequantize", hv.QUANTIZE),
                                        ("linear", hv.LINEAR), ("fused", hv.FUSED), ("logprobs", hv.LOGPROBS)])
def test_host_validation(codes, name, cases):
    for (kw, want), got in zip(cases, codes[name]):
        assert got == want, (name, kw)


def test_sizes():
    L = binding.lib()
    for rows, cols in ((1, 1), (128, 32), (129, 33), (1000, 4096), (7, 2207)):
        for name, code in (("mx", 0), ("nv", 1)):
            row, scales = binding._fp4_sizes(rows, cols, name)
            assert L.spec_fp4_code_bytes(rows, cols) == rows * row
            assert L.spec_fp4_scale_bytes(rows, cols, code) == scales
    for bad in ((-1, 4), (4, 0), ((1 << 24) + 1, 4), (4, (1 << 24) + 1)):
        assert L.spec_fp4_code_bytes(*bad) == 0 and L.spec_fp4_scale_bytes(*bad, 0) == 0
    assert L.spec_fp4_scale_bytes(4, 4, 2) == 0
    size = L.spec_draft_fused_fp4_workspace_size
    assert size(640, 1001, 200, 10, 0) % 256 == 0
    assert size(640, 1001, 200, 10, 0) >= 640 * 1008 * 2 + 640 * 112 + 5 * 2 * 512
    for bad in ((0, 9, 9, 1, 0), (1, 0, 9, 1, 0), (1, 9, 0, 1, 0), (1, 9, 9, 0, 0), (1, 9, 9, 10, 0), (1, 9, 9, 1, 2),
                (1, (1 << 21) + 1, 9, 1, 0), ((1 << 24) + 1, 9, 9, 1, 0)):
        assert size(*bad) == 0


class Tensor(FakeTensor):
    def stride(self, i=None):
        return self._strides if i is None else self._strides[i]

    def __getitem__(self, at):
        return self

    def element_size(self):
        return self.dtype.itemsize


class Torch(FakeTorch):
    def empty(self, shape, dtype=None, device=None):
        t = super().empty(shape, dtype, device)
        self.cuda.made[-1] = Tensor(t.shape, t.dtype, t.dev, t.made_on)
        return self.cuda.made[-1]

    def empty_strided(self, shape, strides, dtype=None, device=None):
        t = self.empty(shape, dtype, device)
        t._strides = strides
        return t


class Lib(FakeLib):
    def __getattr__(self, name):
        return (lambda *a: 1024) if "workspace_size" in name else super().__getattr__(name)


@pytest.fixture
def fake(monkeypatch):
    t = Torch()
    monkeypatch.setattr(binding, "torch", t)
    monkeypatch.setattr(binding, "_lib", Lib(t.cuda))
    return t.cuda


def T(shape, dtype, dev=0, **kw):
    return Tensor(shape, dtype, dev, **kw)


def matrix(rows, cols, fmt="mx", dev=0, ts=1.0):
    row, scales = binding._fp4_sizes(rows, cols, fmt)
    return binding.Fp4Matrix(T((rows, row), U8, dev), T((scales,), U8, dev), rows, cols, fmt, ts)


def _calls(dev):
    x, logits = T((5, 64), BF, dev), T((5, 640), F32, dev)
    a, w = matrix(5, 64, dev=dev), matrix(16, 64, dev=dev)
    return {"quantize": lambda s=None: binding.fp4_quantize(x, stream=s),
            "dequantize": lambda s=None: binding.fp4_dequantize(a, stream=s),
            "linear": lambda s=None: binding.fp4_linear(a, w, stream=s),
            "fused": lambda s=None: binding.draft_topk_fused_fp4(x, w, 3, stream=s),
            "logprobs": lambda s=None: binding.token_logprobs(logits, T((5,), I32, dev), 3, stream=s)}


CALLS = ["quantize", "dequantize", "linear", "fused", "logprobs"]


class OtherStream:  # not one of torch's
    cuda_stream = 88


@pytest.mark.parametrize("dev", [0, 1])
@pytest.mark.parametrize("stream", ["none", "current", "side", "other"])
@pytest.mark.parametrize("call", CALLS)
def test_allocations_and_launches_go_to_the_stream(fake, dev, stream, call):
    from test_paged_streams import FakeStream
    fake.streams[dev] = 11
    s = {"none": None, "current": FakeStream(dev, 11), "side": FakeStream(dev, 77), "other": OtherStream()}[stream]
    raw = {"none": 11, "current": 11, "side": 77, "other": 88}[stream]
    _calls(dev)[call](s)
    assert len(fake.calls) == 1 and fake.calls[0][1:] == (dev, raw)
    assert fake.made and all(t.made_on == (dev, raw) for t in fake.made)
    assert fake.current == 0 and fake.streams[dev] == 11


@pytest.mark.parametrize("call", CALLS)
def test_refusals_of_devices(fake, call):
    from test_paged_streams import FakeStream
    with pytest.raises(ValueError):
        _calls(0)[call](FakeStream(1, 77))
    with pytest.raises((ValueError, TypeError)):
        _calls(-1)[call]()
    assert not fake.calls and not fake.made


BAD = {
    "x of whole numbers": lambda: binding.fp4_quantize(T((5, 64), I32)),
    "x of three dimensions": lambda: binding.fp4_quantize(T((5, 2, 64), BF)),
    "x with strided rows": lambda: binding.fp4_quantize(T((5, 64), BF, strides=(128, 2))),
    "another format": lambda: binding.fp4_quantize(T((5, 64), BF), "e2m1"),
    "out of other sizes": lambda: binding.fp4_quantize(T((5, 64), BF), out=matrix(5, 32)),
    "out of another format": lambda: binding.fp4_quantize(T((5, 64), BF), out=matrix(5, 64, "nv")),
    "out of another scale": lambda: binding.fp4_quantize(T((5, 64), BF), "nv", 1.0, out=matrix(5, 64, "nv", 0, 2.0)),
    "out on another device": lambda: binding.fp4_quantize(T((5, 64), BF), out=matrix(5, 64, dev=1)),
    "codes of another size": lambda: binding.fp4_dequantize(matrix(5, 64)._replace(rows=6)),
    "scales of another size": lambda: binding.fp4_dequantize(matrix(128, 128)._replace(scales=T((1,), U8))),
    "codes of another type": lambda: binding.fp4_dequantize(matrix(5, 64)._replace(codes=T((5, 32), I32))),
    "codes of another format": lambda: binding.fp4_dequantize(matrix(5, 64)._replace(format="fp8")),
    "no columns": lambda: binding.fp4_dequantize(matrix(5, 64)._replace(cols=0)),
    "half precision values": lambda: binding.fp4_dequantize(matrix(5, 64), torch.float16),
    "values elsewhere": lambda: binding.fp4_dequantize(matrix(5, 64), out=T((5, 64), BF, 1)),
    "values of another type": lambda: binding.fp4_dequantize(matrix(5, 64), out=T((5, 64), F32)),
    "values of another size": lambda: binding.fp4_dequantize(matrix(5, 64), out=T((5, 65), BF)),
    "values in columns": lambda: binding.fp4_dequantize(matrix(5, 64), out=T((5, 64), BF, strides=(1, 5))),
    "two formats": lambda: binding.fp4_linear(matrix(5, 64), matrix(16, 64, "nv")),
    "two lengths": lambda: binding.fp4_linear(matrix(5, 64), matrix(16, 32)),
    "two devices": lambda: binding.fp4_linear(matrix(5, 64), matrix(16, 64, dev=1)),
    "a result elsewhere": lambda: binding.fp4_linear(matrix(5, 64), matrix(16, 64), out=T((5, 16), BF, 1)),
    "a result of another size": lambda: binding.fp4_linear(matrix(5, 64), matrix(16, 64), out=T((16, 5), BF)),
    "a result of half precision": lambda: binding.fp4_linear(matrix(5, 64), matrix(16, 64), torch.float16),
    "fp32 features": lambda: binding.draft_topk_fused_fp4(T((5, 64), F32), matrix(16, 64), 2),
    "features of another length": lambda: binding.draft_topk_fused_fp4(T((5, 32), BF), matrix(16, 64), 2),
    "a head elsewhere": lambda: binding.draft_topk_fused_fp4(T((5, 64), BF), matrix(16, 64, dev=1), 2),
    "a workspace elsewhere": lambda: binding.draft_topk_fused_fp4(T((5, 64), BF), matrix(16, 64), 2,
                                                                  workspace=T((4096,), U8, 1)),
    "logits of half precision": lambda: binding.token_logprobs(T((5, 64), torch.float16), None, 1),
    "logits of three dimensions": lambda: binding.token_logprobs(T((5, 2, 64), BF), None, 1),
    "logits in columns": lambda: binding.token_logprobs(T((5, 64), BF, strides=(1, 8)), None, 1),
    "tokens of 64 bits": lambda: binding.token_logprobs(T((5, 64), BF), T((5,), torch.int64)),
    "tokens of another number": lambda: binding.token_logprobs(T((5, 64), BF), T((4,), I32)),
    "tokens elsewhere": lambda: binding.token_logprobs(T((5, 64), BF), T((5,), I32, 1)),
    "tokens of three dimensions": lambda: binding.token_logprobs(T((5, 64), BF), T((5, 1, 1), I32)),
    "rows of 64 bits": lambda: binding.token_logprobs(T((5, 64), BF), None, 1, rows=T((2,), torch.int64)),
    "rows of two dimensions": lambda: binding.token_logprobs(T((5, 64), BF), None, 1, rows=T((2, 1), I32)),
}


@pytest.mark.parametrize("name", BAD)
def test_the_binding_refuses(fake, name):
    with pytest.raises((TypeError, ValueError)):
        BAD[name]()
    assert not fake.calls


def test_padded_results(fake):
    cuda = torch.device("cuda", 0)
    assert binding._padded(3, 9, BF, cuda) is fake.made[-1]
    assert fake.made[-1].shape == (3, 9) and fake.made[-1].stride() == (16, 1)
    assert binding._padded(3, 9, F32, cuda).stride() == (12, 1)
    assert binding._padded(3, 8, F32, cuda).stride() == (8, 1)
    # a result with padded rows goes to the kernel with its pitch, one row with any
    assert binding._pitch(binding._padded(3, 9, F32, cuda), 9) == 12
    assert binding._pitch(T((1, 9), F32, strides=(77, 1)), 9) == 12
