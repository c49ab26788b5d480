"""The head's calls one after another, as a decoding round makes them: draft features through a 4-bit head
and its ranking, the target's logits from a 4-bit head into the verify step, the log probabilities of the
tokens it emits by their rows; eager, captured and replayed, on side streams."""
import numpy as np
import pytest
import torch

from oracle import fp4 as oracle_fp4
from oracle.draft import draft_topk as oracle_draft
from oracle.logprobs import token_logprobs as oracle_logprobs
from speculative_decoding_tree_spec_gb300 import binding
from speculative_decoding_tree_spec_gb300 import workloads as wl

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
SCALES = {"mx": (1.0, 1.0), "nv": (2.0 ** -4, 2.0 ** -10)}


def _features(R, d, seed):
    return torch.randn((R, d), generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV).to(BF)


def _head(V, d, fmt, seed=1):
    w = torch.randn((V, d), generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV) * 0.02
    return binding.fp4_quantize(w.to(BF), fmt, SCALES[fmt][1])


def _bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("R,V,d", [(1, 1000, 64), (10, 4001, 512), (130, 2500, 1024), (640, 1003, 128)])
def test_draft_head_in_four_bits(fmt, R, V, d):
    """One call gives what its three steps give, and what the oracle ranks on those logits."""
    x, head = _features(R, d, R), _head(V, d, fmt)
    a = binding.draft_topk_fused_fp4(x, head, 10, 0.8, SCALES[fmt][0], want_logits=True)
    b = binding.draft_topk_fused_fp4(x, head, 10, 0.8, SCALES[fmt][0])
    logits = binding.fp4_linear(binding.fp4_quantize(x, fmt, SCALES[fmt][0]), head)
    c = binding.draft_topk(logits, 10, 0.8)
    torch.cuda.synchronize()
    assert torch.equal(a["logits"], logits)
    for key in ("tokens", "probs", "status"):
        assert torch.equal(a[key], b[key]) and torch.equal(a[key], c[key])
    tok, prob, st = oracle_draft(_bits(logits)[:5], 10, 0.8)
    assert a["tokens"][:5].cpu().tolist() == tok.tolist() and not st.any()
    assert (np.abs(a["probs"][:5].cpu().numpy() - prob) <= 1e-5 * prob).all()
    # the logits are the product of what codes and scales stand for, rounded once
    q = binding.fp4_quantize(x, fmt, SCALES[fmt][0])
    av, wv = (binding.fp4_dequantize(m, F32).double() for m in (q, head))
    want, size = av @ wv.T, av.abs() @ wv.abs().T
    assert ((logits.double() - want).abs() <= size * d * 2.0 ** -23 + want.abs() * 2.0 ** -8).all()


def _round(fmt, B=6, N=12, V=2000, d=256):
    """The inputs of a verify step whose target logits come from features."""
    w = wl.WORKLOADS["tree60_b64_v128256"].with_(B=B, N=N, V=V, depth=4, temperature=0.9, top_p=1.0)
    inp = wl.build_inputs(w, seed=3, device=torch.device(DEV))
    return {"x": _features(B * N, d, 9), "head": _head(V, d, fmt, 5), "q": inp["q"],
            "tokens": torch.as_tensor(inp["tokens"], device=DEV),
            "parents": torch.as_tensor(inp["parents"], device=DEV), "depth": inp["max_depth"], "B": B, "N": N,
            "V": V, "fmt": fmt}


def _step(s, logits):
    """Features to reported log probabilities; logits [B N, V] is written."""
    B, N, V = s["B"], s["N"], s["V"]
    binding.fp4_linear(binding.fp4_quantize(s["x"], s["fmt"], SCALES[s["fmt"]][0]), s["head"], alpha=4.0, out=logits)
    res = binding.verify_tree(logits.view(B, N, V), s["q"], s["tokens"], s["parents"], s["depth"], 0.9, seed=11)
    first = torch.arange(B, device=DEV, dtype=I32)[:, None] * N
    rows = torch.where(res["path"] >= 0, first + res["path"], -1).view(-1)
    lp = binding.token_logprobs(logits, res["tokens"].view(-1), 4, 0.9, rows=rows)
    return res, rows, lp


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_round(fmt):
    s = _round(fmt)
    logits = torch.empty((s["B"] * s["N"], s["V"]), dtype=BF, device=DEV)
    res, rows, lp = _step(s, logits)
    torch.cuda.synchronize()
    assert not res["status"].any()
    tokens = res["tokens"].view(-1).cpu().numpy()
    want = oracle_logprobs(_bits(logits), tokens[:, None], 4, 0.9, rows.cpu().numpy())
    assert (rows.cpu().numpy() >= 0).sum() == int((res["accept_len"] + 1).sum())
    np.testing.assert_array_equal(lp["status"].cpu().numpy(), want["status"])
    np.testing.assert_array_equal(lp["top_tokens"].cpu().numpy(), want["top_tokens"])
    got = lp["logprobs"].cpu().numpy()
    real = rows.cpu().numpy() >= 0
    assert np.isfinite(got[real]).all() and np.isneginf(got[~real]).all()
    # weights 2^a, |a| <= log2 V + 30, are off by 2 |a| 2^-24 + 2^-22 at most (test_gpu_logprobs.py)
    tol = (41 * 2 + 4 + 8) * 2.0 ** -24 * (1 + np.abs(got))
    assert (np.abs(got - want["logprobs"][:, 0]) <= tol)[real].all()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_round_captured_and_replayed(fmt):
    """A captured round replayed on new features gives what an eager one gives."""
    s = _round(fmt)
    logits = torch.empty((s["B"] * s["N"], s["V"]), dtype=BF, device=DEV)
    _step(s, logits)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        res, rows, lp = _step(s, logits)
    for seed in (21, 22):
        s["x"].copy_(_features(*s["x"].shape, seed))
        g.replay()
        torch.cuda.synchronize()
        got = {**{k: v.clone() for k, v in res.items()}, **{"l_" + k: v.clone() for k, v in lp.items()}}
        r2, _, l2 = _step(s, logits)
        torch.cuda.synchronize()
        for k, v in {**r2, **{"l_" + k: v for k, v in l2.items()}}.items():
            assert torch.equal(got[k].nan_to_num(), v.nan_to_num()), k


def test_two_streams_at_once():
    """Calls of two streams, each with its own sizes, between those of the default stream."""
    jobs = []
    for i, (fmt, R, V, d) in enumerate((("mx", 3, 9000, 2048), ("nv", 200, 3000, 1024))):
        x, head = _features(R, d, i), _head(V, d, fmt, i)
        t = torch.randint(0, V, (R,), device=DEV, dtype=I32)
        def job(stream=None, x=x, head=head, fmt=fmt, t=t):
            q = binding.fp4_quantize(x, fmt, SCALES[fmt][0], stream=stream)
            z = binding.fp4_linear(q, head, F32, stream=stream)
            r = binding.token_logprobs(z, t, 7, stream=stream)
            return [z, binding.fp4_dequantize(q, stream=stream), *r.values(),
                    *binding.draft_topk_fused_fp4(x, head, 5, 1.0, SCALES[fmt][0], stream=stream).values()]
        jobs.append(job)
    want = [j() for j in jobs]
    side = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for _ in range(40):
        got = []
        for s, j in zip(side, jobs):
            j(s)
            got.append(j(s))
            torch.full((1 << 24,), float("nan"), device=DEV)  # the next owner of the default stream's memory
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))


def test_values_that_overlap_nothing_are_left():
    """A result within a larger matrix: only its rows and columns are written."""
    x, head = _features(70, 128, 1), _head(200, 128, "mx", 2)
    q = binding.fp4_quantize(x)
    big = torch.full((90, 256), 5.0, dtype=F32, device=DEV)
    binding.fp4_linear(q, head, F32, out=big[10:80, 8:208])
    torch.cuda.synchronize()
    assert torch.equal(big[10:80, 8:208], binding.fp4_linear(q, head, F32))
    keep = torch.ones_like(big, dtype=torch.bool)
    keep[10:80, 8:208] = False
    assert (big[keep] == 5).all()


def test_oracle_values_of_a_device_matrix():
    """unpack reads what the device wrote."""
    q = binding.fp4_quantize(_features(131, 80, 4)[:, :77], "nv", 0.25)  # rows on 16-byte boundaries
    codes, scales = oracle_fp4.unpack(q.codes.cpu().numpy(), q.scales.cpu().numpy(), 131, 77, "nv")
    got = binding.fp4_dequantize(q, F32).cpu().numpy()
    np.testing.assert_array_equal(got, oracle_fp4.values(codes, scales, "nv", 0.25).astype(np.float32))
