"""Lengths beyond the positions that a page table can hold are refused (the calls run in a child
process that sees no GPU: tests/paged_limit_cases.py)."""
import json
import os
import subprocess
import sys

import __graft_entry__
import paged_limit_cases as pl

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_shared_lengths_beyond_the_positions_are_refused():
    __graft_entry__.build()
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    env["PYTHONPATH"] = os.pathsep.join([ROOT, here, env.get("PYTHONPATH", "")])
    r = subprocess.run([sys.executable, os.path.join(here, "paged_limit_cases.py")],
                       capture_output=True, text=True, env=env, cwd=ROOT, timeout=300)
    assert r.returncode == 0, r.stderr
    got = json.loads(r.stdout)
    assert got["attend"] == [want for _, want in pl.SHARED]
    assert got["size"] == [0] * len(pl.SHARED) and got["size_in_range"] > 0
