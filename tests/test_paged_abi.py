"""The paged-cache entry points refuse bad arguments on the host, before anything is launched
(the calls run in a child process that sees no GPU: tests/paged_validation_cases.py)."""
import ctypes
import json
import os
import subprocess
import sys

import pytest

import __graft_entry__
import paged_validation_cases as pv
from speculative_decoding_tree_spec_gb300 import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def codes():
    __graft_entry__.build()
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    env["PYTHONPATH"] = os.pathsep.join([ROOT, here, env.get("PYTHONPATH", "")])
    r = subprocess.run([sys.executable, os.path.join(here, "paged_validation_cases.py")],
                       capture_output=True, text=True, env=env, cwd=ROOT, timeout=300)
    assert r.returncode == 0, r.stderr
    return json.loads(r.stdout)


@pytest.mark.parametrize("name,cases", [("append", pv.APPEND), ("attend", pv.ATTEND),
                                        ("commit", pv.COMMIT)])
def test_host_validation(codes, name, cases):
    for (kw, want), got in zip(cases, codes[name]):
        assert got == want, (name, kw)


def test_struct_sizes():
    assert ctypes.sizeof(binding.PagedLayout) == 40
    assert ctypes.sizeof(binding.NodeLayout) == 24


def test_workspace_size():
    size = binding.tree_attention_workspace_size
    a = size(64, 60, 32, 8, 128)
    assert a > 0 and a % 256 == 0
    # the shared positions' result: one fp32 row and one statistic per query
    assert size(64, 60, 32, 8, 128, 64) >= a + 64 * 60 * 32 * (128 + 1) * 4
    for bad in ((-1, 1, 8, 8, 64), (1, 1, 8, 3, 64), (1, 1, 8, 8, 136), (1, 1, 8, 8, 0),
                (1 << 20, 1 << 10, 8, 8, 64), (1, 1, 8, 8, 64, -1)):
        assert size(*bad) == 0, bad
