"""4-bit matrices and products beyond 2^31 bytes and elements, a head with a scale of its own, and calls
joined from two streams, eager and captured.  Everything is compared bit for bit: with the same call on
the far part alone, or with the same calls in one stream."""
import numpy as np
import pytest
import torch

from speculative_decoding_tree_spec_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
TS = {"mx": 1.0, "nv": 2.0 ** -10}


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_codes_beyond_2_to_the_31(fmt):
    """2.25 GB of codes, 9 GB of values: the last rows as a matrix of their own."""
    R, K, tail = 128 * 8600, 4096, 128 * 3
    x = torch.zeros((R, K), dtype=BF, device=DEV)
    x[-tail:] = torch.randn((tail, K), generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).to(BF)
    q, part = binding.fp4_quantize(x, fmt, TS[fmt]), binding.fp4_quantize(x[-tail:], fmt, TS[fmt])
    del x
    assert q.codes.numel() > 2 ** 31
    assert torch.equal(q.codes[-tail:], part.codes) and not q.codes[:-tail].any()
    assert torch.equal(q.scales[-part.scales.numel():], part.scales)
    back = binding.fp4_dequantize(q, BF)
    assert torch.equal(back[-tail:], binding.fp4_dequantize(part, BF)) and not back[:-tail].any()
    del back
    a = binding.fp4_quantize(torch.randn((5, K), device=DEV).to(BF), fmt, TS[fmt])
    out = binding.fp4_linear(a, q, F32)
    # the far rows in the same tiles and in the same order of K
    assert torch.equal(out[:, -tail:], binding.fp4_linear(a, _rows(q, R - 128 * 400), F32)[:, -tail:])
    assert not out[:, :-tail].any()


def _rows(m, first):
    """The rows from `first`, a multiple of 128, on."""
    return m._replace(codes=m.codes[first:], scales=m.scales[m.scales.numel() // (m.rows // 128) * (first // 128):],
                      rows=m.rows - first)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_results_beyond_2_to_the_31(dtype):
    R, V, K = 17000, 128256, 64
    g = torch.Generator(device=DEV).manual_seed(2)
    a = binding.fp4_quantize(torch.randn((R, K), generator=g, device=DEV).to(BF))
    w = binding.fp4_quantize(torch.randn((V, K), generator=g, device=DEV).to(BF))
    out = binding.fp4_linear(a, w, dtype)
    assert out.numel() > 2 ** 31
    av, wv = binding.fp4_dequantize(a, F32), binding.fp4_dequantize(w, F32)
    for r in (0, 8191, 16384, R - 1):
        want = av[r].double() @ wv.double().T
        size = av[r].double().abs() @ wv.double().abs().T
        tol = size * K * 2.0 ** -23 + want.abs() * torch.finfo(dtype).eps / 2 * 1.01
        assert ((out[r].double() - want).abs() <= tol).all()


@pytest.mark.parametrize("scale", [0.0123, 3.0, 1e-20])
def test_a_head_with_a_scale_of_its_own(scale):
    """The draft call on a head whose tensor scale is no power of two: as its three steps."""
    x = torch.randn((30, 256), generator=torch.Generator(device=DEV).manual_seed(3), device=DEV).to(BF)
    head = binding.fp4_quantize(torch.randn((3001, 256), device=DEV).to(BF), "nv", 0.25)
    head = head._replace(tensor_scale=float(np.float32(scale)))
    got = binding.draft_topk_fused_fp4(x, head, 6, 0.9, 2.0 ** -4, want_logits=True)
    logits = binding.fp4_linear(binding.fp4_quantize(x, "nv", 2.0 ** -4), head)
    want = binding.draft_topk(logits, 6, 0.9)
    assert torch.equal(got["logits"], logits) and logits.any()
    assert all(torch.equal(got[k], want[k]) for k in want) and not got["status"].any()


def _joined(x, wt, side):
    """The weight quantised on another stream, joined before the product."""
    main = torch.cuda.current_stream()
    side.wait_stream(main)
    w = binding.fp4_quantize(wt, stream=side)
    a = binding.fp4_quantize(x)
    main.wait_stream(side)
    w.codes.record_stream(main)
    w.scales.record_stream(main)
    return binding.fp4_linear(a, w, F32)


@pytest.mark.parametrize("R,V,K", [(3, 40000, 2048), (200, 20000, 512), (5, 512, 4096)])
def test_products_behind_two_streams(R, V, K):
    g = torch.Generator(device=DEV).manual_seed(R)
    x, wt = (torch.randn((n, K), generator=g, device=DEV).to(BF) for n in (R, V))
    side = torch.cuda.Stream()

    def want():
        return binding.fp4_linear(binding.fp4_quantize(x), binding.fp4_quantize(wt), F32)

    for _ in range(10):
        assert torch.equal(_joined(x, wt, side), want())
        wt.neg_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _joined(x, wt, side)
    for seed in range(3):
        x.copy_(torch.randn((R, K), generator=g, device=DEV))
        wt.copy_(torch.randn((V, K), generator=g, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want())
