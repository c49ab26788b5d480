"""Values at the ends of the head calls' ranges that the host has to refuse.  Run as a script in a child
process that sees no GPU: a call that is not refused ends with the launch's error (-5), or with 0 where
it has no rows.  Prints the return codes as JSON."""
import json
import sys

import head_validation_cases as hv
from speculative_decoding_tree_spec_gb300 import binding

# feature scale, weight scale: their product is the logits' factor, a float32
SCALES = [
    (dict(feature_scale=2.0 ** -100, weight_scale=2.0 ** -50), -1),
    (dict(feature_scale=2.0 ** -75, weight_scale=2.0 ** -75), -1),
    (dict(feature_scale=2.0 ** -100, weight_scale=2.0 ** -100), -1),
    (dict(feature_scale=2.0 ** 100, weight_scale=2.0 ** 28), -1),
    (dict(feature_scale=2.0 ** -100, weight_scale=2.0 ** -49, R=0), 0),
    (dict(feature_scale=2.0 ** -63, weight_scale=2.0 ** -63, R=0), 0),
    (dict(feature_scale=2.0 ** 100, weight_scale=2.0 ** 27, R=0), 0),
    (dict(feature_scale=2.0 ** 100, weight_scale=2.0 ** -100, R=0), 0),
    # a weight's scale is a factor of the logits, and need not be a power of two
    (dict(feature_scale=2.0 ** -4, weight_scale=0.0123, R=0), 0),
    (dict(weight_scale=3e-38, R=0), 0),
    (dict(weight_scale=1e38, R=0), 0),
    (dict(feature_scale=4.0, weight_scale=1e38), -1),
    (dict(feature_scale=2.0 ** -30, weight_scale=0.3e-37), -1),
    (dict(weight_scale=-0.5), -1),
    (dict(weight_scale=float("nan")), -1),
    (dict(weight_scale=float("inf")), -1),
]

# given tokens per row: the kernels count them in 32 bits, a block's threads past the last
GIVEN = [
    (dict(G=2 ** 31 - 1), -6),
    (dict(G=2 ** 31 - 200), -6),
    (dict(G=2 ** 30 + 1), -6),
    (dict(G=2 ** 30, R=0), 0),
]


def main():
    L = binding.lib()
    print(json.dumps({"scales": [hv.fused(L, format=1, **kw) for kw, _ in SCALES],
                      "given": [hv.logprobs(L, **kw) for kw, _ in GIVEN]}))


if __name__ == "__main__":
    sys.exit(main())
