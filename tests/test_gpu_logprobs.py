"""Token log probabilities, entropy and top alternatives against the oracle in 64 bits.

Tolerances, from the arithmetic (u = 2^-24): x = (z - max) / T takes a rounded difference and a rounded
product (2 u |x|); a weight 2^a is off by |a| u (a's rounding, twice) plus 2^-22 (the exponential);
ln S is off by what its weights are, relatively, plus a few u of itself, the entropy by that and by as
much of the mean of |x|; the results are rounded in fp32.  Where p is spread over n tokens, |a| in the
sums that matter is below log2 n + 30 (smaller weights are below 2^-30 of the sum)."""
import numpy as np
import pytest
import torch

from oracle.logprobs import token_logprobs as oracle_logprobs
from speculative_decoding_tree_spec_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def _rows(x, dtype):
    per = 16 // torch.empty((), dtype=dtype).element_size()
    R, V = x.shape
    d = torch.full((R, -(-V // per) * per), 50.0, dtype=dtype, device=DEV)[:, :V]
    d.copy_(x.to(dtype))
    return d


def _check(x, dtype, tokens=None, k=5, T=1.0, rows=None):
    d = _rows(x, dtype)
    t = None if tokens is None else torch.as_tensor(tokens, dtype=torch.int32, device=DEV)
    i = None if rows is None else torch.as_tensor(rows, dtype=torch.int32, device=DEV)
    got = binding.token_logprobs(d, t, k, T, rows=i)
    torch.cuda.synchronize()
    host = d.float().cpu().numpy()
    want = oracle_logprobs(host, None if t is None else t.cpu().numpy(), k, T, rows)
    g = {n: v.cpu().numpy() for n, v in got.items()}
    np.testing.assert_array_equal(g["status"], want["status"])
    np.testing.assert_array_equal(g["top_tokens"], want["top_tokens"])
    n_bits = np.log2(x.shape[1]) + 30
    weight = n_bits * 2 * U + 2.0 ** -22  # relative, of one weight and so of S
    for name in ("logprobs", "top_logprobs"):
        w = want[name].reshape(g[name].shape)
        np.testing.assert_array_equal(np.isnan(g[name]), np.isnan(w))
        np.testing.assert_array_equal(np.isneginf(g[name]), np.isneginf(w))
        f = np.isfinite(w)
        # ln S is at most |w| or, where w is near 0, S - 1 at most about |w|
        tol = np.abs(w) * (weight + 8 * U) + np.minimum(np.abs(w), 1.0) * weight
        tol += np.log2(x.shape[1]) * 8 * U
        assert (np.abs(g[name] - w)[f] <= tol[f]).all(), (name, np.abs(g[name] - w)[f].max())
    w = want["entropy"]
    np.testing.assert_array_equal(np.isnan(g["entropy"]), np.isnan(w))
    f = np.isfinite(w)
    tol = weight * (1 + 2 * np.abs(w)) + 16 * U * np.abs(w)
    assert (np.abs(g["entropy"] - w)[f] <= tol[f]).all(), np.abs(g["entropy"] - w)[f].max()
    return got


def _gauss(R, V, seed, std=3.0):
    return torch.randn((R, V), generator=torch.Generator().manual_seed(seed)) * std


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("V", [1, 2, 31, 32, 33, 255, 257, 1000, 1024, 1025, 2047, 4096 + 3, 9001, 32000, 128256])
def test_vocabularies(dtype, V):
    R = 5
    g = np.random.default_rng(V)
    _check(_gauss(R, V, V), dtype, g.integers(0, V, (R, 2)), min(V, 10))


@pytest.mark.parametrize("k", [0, 1, 2, 7, 20, 32])
@pytest.mark.parametrize("V", [40, 900, 5000, 70001])
def test_numbers_of_alternatives(k, V):
    _check(_gauss(9, V, k + V), BF, np.arange(9) % V, k)
    _check(_gauss(9, V, k + V), F32, None, k)


@pytest.mark.parametrize("R", [1, 2, 19, 38, 77, 153, 310, 700])
def test_numbers_of_rows(R):
    """One CTA to eight per row."""
    g = np.random.default_rng(R)
    _check(_gauss(R, 20000, R), BF, g.integers(0, 20000, R), 10)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("R,V", [(4000, 33), (4000, 300), (3000, 1000), (5000, 1100), (5000, 2000), (2000, 5000)])
def test_many_short_rows(R, V, dtype):
    """Rows by the thousand, a warp or two each: the alternatives against a stable sort."""
    d = _rows(_gauss(R, V, R + V), dtype)
    order = torch.sort(d.float(), dim=1, descending=True, stable=True)[1]
    for k in (1, 3, 4, 17, 32):
        got = binding.token_logprobs(d, order[:, :2].to(torch.int32).contiguous(), k)
        assert torch.equal(got["top_tokens"], order[:, :k].to(torch.int32)) and not got["status"].any()
        n = min(k, 2)
        assert torch.equal(got["top_logprobs"][:, :n], got["logprobs"][:, :n])


@pytest.mark.parametrize("T", [1e-3, 0.25, 0.7, 2.0, 100.0])
@pytest.mark.parametrize("V", [500, 20000])
def test_temperatures(T, V):
    _check(_gauss(6, V, 5), F32, np.arange(6), 5, T)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("V", [700, 30011])
@pytest.mark.parametrize("kind", ["constant", "two levels", "ascending", "descending", "few"])
def test_ties_and_orders(dtype, V, kind):
    if kind == "constant":
        x = torch.full((3, V), 1.25)
    elif kind == "two levels":
        x = (torch.rand((3, V), generator=torch.Generator().manual_seed(4)) < 0.01).float()
    elif kind == "few":
        x = torch.randint(-5, 6, (3, V), generator=torch.Generator().manual_seed(4)).float() / 2
    else:
        x = torch.linspace(-8, 8, V).repeat(3, 1) * (1 if kind == "ascending" else -1)
    for k in (1, 10, 32):
        _check(x, dtype, np.array([[0, 5], [V - 1, 2], [3, 3]]), k)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("V", [100, 1000, 12345])
def test_masked_logits(dtype, V):
    """-inf and the type's lowest number in most places; fewer tokens left than are asked for."""
    x = _gauss(8, V, 8)
    drop = torch.rand((8, V), generator=torch.Generator().manual_seed(9)) < 0.97
    drop[:, 17] = False
    x[drop] = float("-inf")
    x[2, drop[2]] = torch.finfo(dtype).min
    x[3] = float("-inf")
    x[3, V - 1] = -4.0
    _check(x, dtype, np.tile([17, 0, V - 1], (8, 1)), 20)


@pytest.mark.parametrize("V", [64, 800, 25000])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_rows_that_are_not_finite(dtype, V):
    x = _gauss(7, V, 2)
    x[1, V // 3] = float("nan")
    x[2, V - 1] = float("inf")
    x[3] = float("-inf")
    x[4, 0] = float("-inf")
    x[5, 1], x[5, 2] = float("inf"), float("nan")
    _check(x, dtype, np.zeros((7, 1), dtype=int), 3)


def test_one_token_holds_nearly_all():
    """ln p of a token that holds all but a trillionth.  In a wide row a lane adds the 32 weights (fp32: 16)
    of a chunk in fp32 before they join the compensated sum.  In the lane that holds the maximum up to
    31 others are added to its 1 there, and vanish where they are below 2^-24: S then lacks at most 31
    of the other weights, each exp(-gap) here, and ln S is off by at most that; the rest of the
    arithmetic is relative."""
    for V in (32, 1024, 40000):
        x = torch.zeros((2, V))
        x[0, V // 2] = 28.0 + float(np.log(V))
        x[1, 3] = 60.0
        d = _rows(x, F32)
        got = binding.token_logprobs(d, torch.tensor([V // 2, 3], dtype=torch.int32, device=DEV), 1)
        want = oracle_logprobs(d.cpu().numpy(), np.array([[V // 2], [3]]), 1)
        gap = np.array([float(x[0].max()), 60.0])
        lost = 31 * np.exp(-gap) if V > 1024 else 0.0
        for name, w in (("logprobs", want["logprobs"][:, 0]), ("entropy", want["entropy"])):
            off = np.abs(got[name].cpu().numpy() - w)
            # the entropy holds each lost weight times 1 + gap
            assert (off <= 1e-5 * np.abs(w) + lost * (1 if name == "logprobs" else 1 + gap)).all()


@pytest.mark.parametrize("V", [300, 21000])
def test_row_numbers(V):
    """Any order, the same row twice, rows that are not there; tokens that are not there."""
    rows = np.array([5, 0, 5, -1, 11, 12, 3, -2147483648, 2147483647, 5])
    tokens = np.array([[1, -1], [V, 0], [2, V - 1], [0, 0], [5, 5], [1, 2], [-7, 2147483647], [1, 1], [1, 1], [1, 0]])
    got = _check(_gauss(12, V, 3), BF, tokens, 4, 1.0, rows)
    assert got["logprobs"][0, 0] == got["logprobs"][9, 0]


def test_many_given_tokens():
    g = np.random.default_rng(0)
    _check(_gauss(3, 5000, 1), F32, g.integers(0, 5000, (3, 1000)), 0)
    _check(_gauss(3, 500, 1), BF, g.integers(0, 500, (3, 1000)), 2)


def test_wide_vocabulary():
    V = binding.SPEC_MAX_VOCAB
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn((2, V), generator=g, device=DEV)
    x[0, V - 1] = 9.0
    x[1, [5, V // 2]] = 9.0
    _check(x, F32, np.array([V - 1, 5]), 32)


def test_far_rows():
    """Rows more than 2^31 elements from the first."""
    n, V = 17000, 128256
    d = torch.zeros((n, V), dtype=BF, device=DEV)
    d[n - 1] = torch.randn(V, device=DEV).to(BF)
    got = binding.token_logprobs(d, torch.tensor([7], dtype=torch.int32, device=DEV), 5,
                                 rows=torch.tensor([n - 1], dtype=torch.int32, device=DEV))
    want = binding.token_logprobs(d[n - 1:].clone(), torch.tensor([7], dtype=torch.int32, device=DEV), 5)
    assert all(torch.equal(got[m], want[m]) for m in got)


def test_empty():
    got = binding.token_logprobs(torch.empty((0, 64), device=DEV), None, 3)
    assert got["top_tokens"].shape == (0, 3) and got["entropy"].shape == (0,)
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    got = binding.token_logprobs(torch.randn((4, 64), device=DEV), none, 3, rows=none)
    assert got["logprobs"].shape == (0,)
