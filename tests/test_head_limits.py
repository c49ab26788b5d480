"""The ends of the head calls' ranges: what the host has to refuse (the C calls run in a child process
that sees no GPU: tests/head_limit_cases.py)."""
import ctypes
import json
import os
import subprocess
import sys

import pytest

import __graft_entry__
import head_limit_cases as hl
from speculative_decoding_tree_spec_gb300 import binding
from test_head_abi import fake, matrix  # noqa: F401 (a fixture)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def codes():
    __graft_entry__.build()
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    env["PYTHONPATH"] = os.pathsep.join([ROOT, here, env.get("PYTHONPATH", "")])
    r = subprocess.run([sys.executable, os.path.join(here, "head_limit_cases.py")], capture_output=True,
                       text=True, env=env, cwd=ROOT, timeout=300)
    assert r.returncode == 0, r.stderr
    return json.loads(r.stdout)


def test_scales_whose_product_is_no_float(codes):
    assert codes["scales"] == [want for _, want in hl.SCALES]


def test_given_tokens_beyond_the_counters(codes):
    assert codes["given"] == [want for _, want in hl.GIVEN]


@pytest.mark.parametrize("alpha,sa,sw", [(1.0, 2.0 ** -100, 2.0 ** -100), (1.0, 2.0 ** -75, 2.0 ** -75),
                                         (1e-20, 2.0 ** -100, 1.0), (-1e-45, 2.0 ** -4, 1.0),
                                         (3.0, 2.0 ** -100, 2.0 ** -50), (1e-300, 2.0 ** -100, 2.0 ** -100)])
def test_the_binding_refuses_factors_that_vanish(fake, alpha, sa, sw):  # noqa: F811
    with pytest.raises(ValueError):
        binding.fp4_linear(matrix(5, 64, "nv", 0, sa), matrix(16, 64, "nv", 0, sw), alpha=alpha)
    assert not fake.calls


@pytest.mark.parametrize("alpha,sa,sw", [(0.0, 1.0, 1.0), (0.0, 2.0 ** -100, 2.0 ** -100), (1.0, 2.0 ** -100, 2.0 ** -49),
                                         (3.0, 2.0 ** -100, 2.0 ** -49), (1e-30, 2.0 ** -20, 1.0), (-0.7, 0.3, 2.0 ** -9),
                                         (2.0 ** 100, 2.0 ** -100, 2.0 ** -100)])
def test_the_binding_takes_factors_that_are_floats(fake, alpha, sa, sw):  # noqa: F811
    binding.fp4_linear(matrix(5, 64, "nv", 0, sa), matrix(16, 64, "nv", 0, sw), alpha=alpha)
    assert len(fake.calls) == 1
    factor = alpha * sa * sw
    assert ctypes.c_float(factor).value == pytest.approx(factor, rel=2.0 ** -24)
