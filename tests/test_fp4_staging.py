"""The staging buffers of the 4-bit product's epilogue.  A warp stages piece c of its results in buffer
c % 2 after a wait that leaves the newest bulk store's read pending, so a buffer is free only if every
piece, of a whole tile or of one at the matrix's edge, commits exactly one group.  The source says what
the two kinds commit; a model of the groups says whether any order of them writes a buffer that a store
still reads."""
import itertools
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "speculative_decoding_tree_spec_gb300", "csrc")


def _text():
    return open(os.path.join(CSRC, "fp4_linear.cu")).read()


def _commits():
    """{helper: groups that a call commits}"""
    out = {}
    for name, body in re.findall(r"__device__ __forceinline__ void (bulk_\w+)\([^)]*\) \{(.*?)\n\}", _text(), re.S):
        out[name] = body.count("cp.async.bulk.commit_group")
    return out


def _branches():
    """The sources of a whole piece's and of an edge piece's store."""
    epilogue = _text().split("// ---------------- epilogue ----------------")[1].split("bulk_store_wait();")[0]
    whole, edge = re.search(r"if \(v0 \+ 32 <= job\.V\) \{(.*?)\n        \} else \{(.*?)\n        \}\n", epilogue, re.S).groups()
    return whole, edge


def _groups(branch):
    return sum(n * len(re.findall(rf"\b{name}\(", branch)) for name, n in _commits().items())


def _safe(pieces, groups, allowed):
    """pieces: their kinds in order.  A store's read ends only when a wait demands it."""
    pending = []  # (buffer read, or None) of each group not known to be done, oldest first
    for c, kind in enumerate(pieces):
        pending = pending[max(0, len(pending) - allowed):]
        if c % 2 in pending:
            return False
        if kind == "whole":
            pending.append(c % 2)
        pending += [None] * (groups[kind] - (kind == "whole"))
    return True


def test_the_model_knows_the_overwrite():
    assert _safe(["whole"] * 9, {"whole": 1, "edge": 1}, 1)
    assert not _safe(["whole", "edge", "edge"], {"whole": 1, "edge": 0}, 1)
    assert not _safe(["whole"] * 3, {"whole": 1, "edge": 1}, 2)


def test_every_piece_commits_one_group():
    whole, edge = _branches()
    groups = {"whole": _groups(whole), "edge": _groups(edge)}
    allowed = re.findall(r"bulk_store_wait_read<(\d+)>\(\)", _text())
    assert len(allowed) == 1 and _text().count("bulk_store(&tm_out") == 1
    assert groups == {"whole": 1, "edge": 1}
    for order in itertools.product(["whole", "edge"], repeat=8):
        assert _safe(order, groups, int(allowed[0])), order
