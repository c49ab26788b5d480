"""The captured traffic that bench.py adds to its roofline belongs to the current sources of the
kernels it names: a change elsewhere in the library does not put it out."""
import pytest

import bench

CAPTURES = [("cluster_walk", w, bench.WALK_SOURCES) for w in ("tree60_b64_v128256", "tree26_b256_v152064")]
CAPTURES += [("row_pass", "tree60_b64_v128256", None), ("row_pass", "tree26_b256_v152064", None)]
CAPTURES += [("draft_topk", "r640_v128256_k10", bench.DRAFT_SOURCES)]


@pytest.mark.parametrize("profile,workload,sources", CAPTURES)
def test_captures_are_current(profile, workload, sources):
    traffic, state = bench.profiled_traffic(workload, profile, sources)
    assert state == "current" and traffic > 0
