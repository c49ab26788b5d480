"""A wait of the 4-bit product that gives up: the call completes, the results that the wait concerns are
NaN, all others exact, and the next call is normal.  Nothing faults or hangs: the self-test leaves out
one fetch, and each wait on it ends after 20 ms."""
import time

import numpy as np
import pytest
import torch

from oracle import fp4 as oracle_fp4
from speculative_decoding_tree_spec_gb300 import binding
from test_gpu_fp4 import _matrix, _random

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def _stalled(a, w, dtype, tile):
    """The result, and the seconds that the call took."""
    out = binding.fp4_linear(a, w, dtype)  # also loads the kernel
    out.fill_(7.0)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    rc = binding.lib().spec_fp4_linear_test_stall(
        a.codes.data_ptr(), a.scales.data_ptr(), w.codes.data_ptr(), w.scales.data_ptr(),
        binding._FP4_FORMATS[a.format], a.rows, w.rows, a.cols, 1.0, out.data_ptr(), binding._float_dtype(dtype),
        binding._pitch(out, w.rows), tile, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    seconds = time.perf_counter() - t0
    assert rc == 0
    return out, seconds


def _check(fmt, dtype, R, V, K, tile, per, weight_rows):
    """per, weight_rows: rows of a tile of the activations and of the weight."""
    a, w = _random(R, K, fmt, R, 0), _random(V, K, fmt, V, 0)
    want = torch.from_numpy(oracle_fp4.linear(oracle_fp4.values(*a, fmt), oracle_fp4.values(*w, fmt))[0])
    want = want.to(F32).to(dtype).to(DEV)  # exact (test_gpu_fp4.py)
    am, wm = _matrix(*a, fmt), _matrix(*w, fmt)
    out, seconds = _stalled(am, wm, dtype, tile)
    lost = torch.zeros((R, V), dtype=torch.bool, device=DEV)
    n_tiles, m_tiles = -(-R // per), -(-V // weight_rows)
    ctas = torch.cuda.get_device_properties(0).multi_processor_count // (weight_rows // 128)
    for t in range(tile, n_tiles * m_tiles, ctas):  # that tile and the later ones of its CTA or pair
        n, m = t % n_tiles, t // n_tiles
        lost[n * per:(n + 1) * per, m * weight_rows:(m + 1) * weight_rows] = True
    assert lost.any() and (V <= weight_rows or not lost.all())
    assert torch.equal(out.isnan(), lost)
    assert torch.equal(out[~lost], want[~lost])
    assert torch.equal(binding.fp4_linear(am, wm, dtype), want)
    return seconds


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("R,V,K,tile,per,weight_rows", [
    (17, 20000, 256, 3, 17, 128),      # single CTAs, one stage, a CTA's next tile as well
    (60, 20100, 2560, 100, 60, 128),   # more steps than stages
    (128, 1000, 512, 7, 128, 128),     # the last tile, which ends inside
    (200, 25000, 1024, 11, 128, 256),  # pairs, two tiles of activations
    (700, 3000, 512, 5, 192, 256),     # pairs, four tiles of activations
    (7, 512, 4096, 2, 7, 128),         # K shared by eight CTAs
    (150, 128, 14336, 0, 150, 128),    # the only tile
    (190, 2000, 14336, 15, 190, 128)])  # K shared, the last tile
def test_a_stage_that_does_not_come(fmt, dtype, R, V, K, tile, per, weight_rows):
    seconds = _check(fmt, dtype, R, V, K, tile, per, weight_rows)
    print(f"{R} x {V} x {K} {fmt}: {seconds * 1e3:.1f} ms")


def test_the_waits_end_in_time():
    """Two waits of 20 ms stand behind each other at most (the products' and the epilogue's run together;
    the fetching warp has nothing of its own under way)."""
    for R, V, K, per, weight_rows in ((60, 20100, 2560, 60, 128), (700, 3000, 512, 192, 256), (7, 512, 4096, 7, 128)):
        seconds = _check("mx", BF, R, V, K, 1, per, weight_rows)
        assert 0.02 <= seconds <= 0.1, seconds


def test_a_draft_row_says_so():
    """The ranking of logits of which some did not come."""
    a, w = _random(9, 64, "mx", 1), _random(600, 64, "mx", 2)
    logits, _ = _stalled(_matrix(*a, "mx"), _matrix(*w, "mx"), BF, 2)
    got = binding.draft_topk(logits, 4)
    assert (got["status"].cpu().numpy() == binding.SPEC_ROW_NONFINITE).all()
    assert (got["tokens"].cpu().numpy() == -1).all()
    lp = binding.token_logprobs(logits, None, 4)
    assert (lp["status"].cpu().numpy() == binding.SPEC_ROW_NONFINITE).all() and np.isnan(lp["entropy"].cpu().numpy()).all()
