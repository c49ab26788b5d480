"""Lengths near 2^31 that the paged calls have to refuse on the host: positions are 32-bit in
the kernels.  Run as a script in a child process that sees no GPU: a call that is not refused ends
with the launch's error.  Prints the return codes as JSON."""
import json
import sys

import paged_validation_cases as pv
from speculative_decoding_tree_spec_gb300 import binding

LIMIT = 0x7FFFF000  # SPEC_MAX_POSITIONS
SHARED = [(LIMIT + 16, -6), (0x7FFFFFF0, -6)]


def main():
    L = binding.lib()
    print(json.dumps({
        "attend": [pv._attend(L, shared_len=n) for n, _ in SHARED],
        "size": [L.spec_tree_attention_workspace_size(2, 2, 4, 2, 64, n, 1) for n, _ in SHARED],
        "size_in_range": L.spec_tree_attention_workspace_size(2, 2, 4, 2, 64, LIMIT, 1)}))


if __name__ == "__main__":
    sys.exit(main())
