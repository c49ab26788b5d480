"""The roofline that bench.py prints for the draft call on a 4-bit head: its operations are held against
four times the bf16 rate and its bytes, the logits among them, against the copy bandwidth; the larger
share is the one reported, and none is above 1 at the call's floor."""
import pytest

import bench

PEAKS = {"hbm_gbs": 6784.8, "bf16_tflops": 1933.1, "bf16_tflops_sustained": 1711.1}


@pytest.mark.parametrize("fmt,scale_bytes", [("mx", 1 / 32), ("nv", 1 / 16)])
@pytest.mark.parametrize("R", [10, 640, 3840])
def test_shares(fmt, scale_bytes, R):
    V, d, k = 128256, 4096, 10
    n_bytes = R * d * 2 + V * d * (0.5 + scale_bytes) + 4 * R * V + R * 84
    flops = 2 * R * V * d
    floor_ms = 1e3 * max(n_bytes / 6784.8e9, flops / (4 * 1933.1e12))
    for ms in (floor_ms, 0.172, 2 * floor_ms):
        r = bench.fp4_head_roofline(R, V, d, k, fmt, ms, PEAKS, "measured")
        assert r["frac"] == pytest.approx(floor_ms / ms, rel=1e-9) and r["frac"] == max(r["frac_hbm"], r["frac_tensor"])
        assert r["frac"] == pytest.approx(r["achieved"] / r["peak"], rel=1e-12)
        assert (r["bound"], r["unit"]) in {("hbm", "GB/s"), ("tensor", "TFLOP/s")}
    assert bench.fp4_head_roofline(R, V, d, k, fmt, floor_ms, PEAKS, "measured")["frac"] <= 1 + 1e-9

