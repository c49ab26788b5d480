"""The log probabilities' launch asks for the shared memory that its kernel uses and no more: a request
made larger to keep CTAs off an SM would suit one share of rows that are not there and slow down the others."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "speculative_decoding_tree_spec_gb300", "csrc")


def test_shared_memory_is_what_the_kernel_uses():
    text = open(os.path.join(CSRC, "logprobs.cu")).read()
    asked = re.findall(r"dynamicSmemBytes\s*=\s*([^;]+);", text)
    # the rings of W warps and four maxima per load
    assert asked == ["(size_t)W * kLpRing + (job.k > 0 ? (size_t)job.n_loads * 16 : 0)"]
