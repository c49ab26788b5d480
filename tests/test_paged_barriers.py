"""Named barriers of the tree attention's kernels: a barrier's number has one thread count, a
number in the source.  (A count that changes from use to use keeps apart only while every wait in
between is honoured; after one that gave up, threads of two uses could meet in one barrier.)"""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "speculative_decoding_tree_spec_gb300", "csrc")


def test_each_named_barrier_has_one_count():
    text = open(os.path.join(CSRC, "attention_tc.cu")).read()
    kinds = {}
    for number, count in re.findall(r"\bhalf_barrier<(\d+), ([^>]+)>\(\)", text):
        kinds.setdefault(number, set()).add(count)
    assert len(kinds) == 2 and all(len(v) == 1 for v in kinds.values()), kinds
    # the template is the only place that issues one
    assert len(re.findall(r"\bbar\.sync\b", text)) == 1 and "named_sync" not in text
