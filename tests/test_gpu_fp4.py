"""Block-scaled 4-bit floating point against the oracle: codes and scales byte for byte, the values
they stand for, and the product of two such matrices.  Every rounding of the quantisation is defined
by the exact quotient, so nothing there has a tolerance."""
import numpy as np
import pytest
import torch

from oracle import fp4 as oracle_fp4
from speculative_decoding_tree_spec_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
TS = {"mx": 1.0, "nv": 2.0 ** -4}


def _host(x):
    return x.float().cpu().numpy()


def _dev_rows(x):
    """On the device with rows on 16-byte boundaries."""
    per = 16 // x.element_size()
    R, K = x.shape
    d = torch.full((R, -(-K // per) * per), 7.0, dtype=x.dtype, device=DEV)[:, :K]
    d.copy_(x)
    return d


def _unsigned_zeros(packed):
    """The sign of a zero says nothing."""
    low, high = packed & 15, packed >> 4
    return np.where(low == 8, 0, low) | (np.where(high == 8, 0, high) << 4)


def _check_quantize(x, fmt, ts):
    R, K = x.shape
    codes, scales = oracle_fp4.quantize(_host(x), fmt, ts)
    want_codes, want_scales = oracle_fp4.pack(codes, scales, fmt)
    d = _dev_rows(x)
    before = d.clone()
    q = binding.fp4_quantize(d, fmt, ts)
    back = {t: binding.fp4_dequantize(q, t) for t in (BF, F32)}
    torch.cuda.synchronize()
    assert torch.equal(d.nan_to_num(), before.nan_to_num())
    got = q.codes.cpu().numpy()
    np.testing.assert_array_equal(q.scales.cpu().numpy(), want_scales)
    np.testing.assert_array_equal(_unsigned_zeros(got), _unsigned_zeros(want_codes))
    values = oracle_fp4.values(codes, scales, fmt, ts)
    for t, v in back.items():
        assert v.shape == (R, K) and v.dtype == t
        want = torch.from_numpy(values).to(F32).to(t)  # exact for these scales
        np.testing.assert_array_equal(_host(v), _host(want))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("R,K", [(1, 1), (1, 32), (3, 17), (5, 33), (129, 64), (33, 255), (2, 520), (130, 100)])
def test_quantize(dtype, fmt, R, K):
    g = torch.Generator().manual_seed(R * 1000 + K)
    x = torch.randn((R, K), generator=g) * torch.exp2(torch.randint(-12, 12, (R, 1), generator=g).float())
    _check_quantize(x.to(dtype), fmt, TS[fmt])


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_quantize_midpoints(fmt):
    """Quotients at the midpoints of two codes and one fp32 step beside them, for scales of every
    significand; block maxima at the midpoints of two scales."""
    rows = []
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=np.float32)
    if fmt == "mx":
        units = 2.0 ** np.arange(-3, 3)
    else:
        units = oracle_fp4.e4m3_values()[list(range(1, 20)) + [60, 61, 62, 63, 126]] * TS["nv"]
    for s in units:
        t = (mids * np.float32(s)).astype(np.float32)
        v = np.concatenate([t, np.nextafter(t, np.float32(0)), np.nextafter(t, np.float32(np.inf))])
        for part in np.array_split(v, 3):
            block = np.zeros(32, dtype=np.float32)
            # the largest element fixes the scale of its block: 6 s (nv), 4 s (mx)
            for h in (0, 16):
                block[h] = 6 * s if fmt == "nv" else 4 * s
                block[h + 1:h + 1 + len(part)] = part
            rows.append(block)
    grid = oracle_fp4.e4m3_values()
    for i in (1, 2, 7, 8, 9, 40, 41, 60, 61, 124, 125):
        m = np.float32((grid[i] + grid[i + 1]) / 2 * 6 * TS["nv"])
        for top in (m, np.nextafter(m, np.float32(0)), np.nextafter(m, np.float32(np.inf))):
            block = np.zeros(32, dtype=np.float32)
            block[[3, 20]] = top
            block[[5, 30]] = -top / 3
            rows.append(block)
    _check_quantize(torch.from_numpy(np.stack(rows)), fmt, TS[fmt])


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_quantize_extremes(fmt, dtype):
    """Zeros, the smallest and the largest numbers, infinities and NaN."""
    x = torch.zeros((12, 96))
    g = torch.Generator().manual_seed(3)
    x[1:] = torch.randn((11, 96), generator=g)
    x[2] *= 1e-38
    x[3] *= 1e38
    x[4] *= 1e-42
    x[5, 40] = float("inf")
    x[6, 70] = float("nan")
    x[7, 3] = float("-inf")
    x[8] = -0.0
    x[9] *= 2.0 ** -14
    x[10] *= 2.0 ** 14
    x[11, 5] = 3.0e38
    _check_quantize(x.to(dtype), fmt, TS[fmt])


@pytest.mark.parametrize("ts", [2.0 ** -100, 2.0 ** -20, 1.0, 2.0 ** 30, 2.0 ** 100])
def test_tensor_scales(ts):
    x = torch.randn((4, 64), generator=torch.Generator().manual_seed(1))
    x[1] *= 2.0 ** -20
    x[2] *= 2.0 ** 30
    x[3] *= 2.0 ** 100
    _check_quantize(x, "nv", ts)


def test_what_lies_beside_the_rows_stays():
    """Outputs are written where the layouts say and nowhere else."""
    x = _dev_rows(torch.randn((70, 45)))
    codes = torch.full((70 * 32 + 64,), 99, dtype=torch.uint8, device=DEV)
    size = 512 * 1 * 1
    scales = torch.full((size + 64,), 99, dtype=torch.uint8, device=DEV)
    m = binding.Fp4Matrix(codes[:70 * 32].view(70, 32), scales[:size], 70, 45, "nv", 0.25)
    assert binding.fp4_quantize(x, "nv", 0.25, out=m) is m
    out = torch.full((70, 56), 3.0, dtype=BF, device=DEV)
    binding.fp4_dequantize(m, BF, out=out[:, :45])
    lin = torch.full((70, 80), 3.0, dtype=F32, device=DEV)
    binding.fp4_linear(m, m, F32, out=lin[:, :70])
    torch.cuda.synchronize()
    assert (codes[70 * 32:] == 99).all() and (scales[size:] == 99).all()
    assert (out[:, 45:] == 3).all() and (lin[:, 70:] == 3).all()


# ---------------------------------------------------------------------------------------
# product
# ---------------------------------------------------------------------------------------
def _random(R, K, fmt, seed, spread=2):
    """Random codes with scales 2^-spread .. 2^spread (nv: with a few significands)."""
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 16, (R, K)).astype(np.uint8)
    blocks = -(-K // oracle_fp4.BLOCK[fmt])
    if fmt == "mx":
        scales = rng.integers(127 - spread, 128 + spread, (R, blocks)).astype(np.uint8)
    else:  # e4m3: exponent 7 is 2^0, significands 1 and 1.5
        e = rng.integers(7 - spread, 8 + spread, (R, blocks))
        scales = (e * 8 + rng.choice([0, 4], (R, blocks))).astype(np.uint8)
    return codes, scales


def _matrix(codes, scales, fmt, ts=1.0):
    packed, tiled = oracle_fp4.pack(codes, scales, fmt)
    return binding.Fp4Matrix(torch.from_numpy(packed).to(DEV), torch.from_numpy(tiled).to(DEV),
                             *codes.shape, fmt, ts)


def _check_exact(R, V, K, fmt, dtype, alpha=1.0, spread=2):
    """Sums of few enough small numbers that no fp32 sum of them, in any order, is rounded: the
    product is exact, and a bf16 result its rounding."""
    a, w = _random(R, K, fmt, R + 3 * V + K, spread), _random(V, K, fmt, R + 5 * V + K, spread)
    av, wv = oracle_fp4.values(*a, fmt), oracle_fp4.values(*w, fmt)
    want, size = oracle_fp4.linear(av, wv, alpha)
    # every product is a multiple of this, and 24 bits hold the sum of all magnitudes
    unit = 0.25 * 2.0 ** (-2 * spread) * (1.0 if fmt == "mx" else 2.0 ** -2)
    assert size.max() / abs(alpha) < unit * 2 ** 24
    got = binding.fp4_linear(_matrix(*a, fmt), _matrix(*w, fmt), dtype, alpha=alpha)
    torch.cuda.synchronize()
    assert got.shape == (R, V) and got.dtype == dtype
    np.testing.assert_array_equal(_host(got), _host(torch.from_numpy(want).to(F32).to(dtype)))


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("R,V,K", [(1, 1, 1), (1, 128, 64), (2, 130, 32), (7, 129, 96), (16, 256, 256), (17, 300, 272),
                                   (33, 128, 512), (64, 257, 320), (65, 255, 300), (96, 128, 256),
                                   (128, 512, 288), (130, 130, 160), (192, 260, 520), (193, 128, 64),
                                   (200, 384, 256), (260, 129, 128), (385, 513, 96), (640, 256, 256)])
def test_linear_exact(fmt, R, V, K):
    _check_exact(R, V, K, fmt, F32)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("R", [1, 48, 200])
def test_linear_rounds_once(fmt, R):
    _check_exact(R, 200, 256, fmt, BF, alpha=0.5)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("R,V,K", [(1, 20000, 1024), (3, 512, 8192), (100, 21000, 512), (700, 20000, 256)],
                         ids=["many tiles", "long", "many pairs", "many of both"])
def test_linear_long(fmt, R, V, K):
    """More tiles than CTAs, and more steps than stages."""
    _check_exact(R, V, K, fmt, F32, spread=0 if K > 1000 else 1)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("R,V,K", [(1, 128, 1024), (1, 1, 2048), (2, 4096, 1024), (5, 200, 2080), (7, 515, 4096), (31, 640, 1100),
                                   (64, 1000, 1500), (65, 130, 2047), (130, 300, 1500), (192, 700, 1056),
                                   (33, 4100, 777)])
def test_linear_of_few_weight_rows(fmt, R, V, K):
    """Tiles whose K several CTAs share: exact whatever the order, in both types."""
    _check_exact(R, V, K, fmt, F32, spread=0)
    _check_exact(R, V, K, fmt, BF, alpha=2.0, spread=0)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_linear_of_extreme_scales(fmt):
    """The smallest scale of one operand against the largest of the other: products that fp32 holds."""
    if fmt == "mx":  # 2^-127 and 2^127; 2^-64 and 2^64
        pairs = [(0, 254), (254, 0), (63, 191), (1, 253)]
    else:  # the smallest subnormal, the largest subnormal, 448
        pairs = [(1, 126), (126, 1), (7, 7), (8, 120), (3, 64)]
    for sa, sw in pairs:
        a, w = _random(20, 192, fmt, sa), _random(150, 192, fmt, sw + 300)
        a[1][:], w[1][:] = sa, sw
        want, _ = oracle_fp4.linear(oracle_fp4.values(*a, fmt), oracle_fp4.values(*w, fmt))
        got = binding.fp4_linear(_matrix(*a, fmt), _matrix(*w, fmt), F32)
        # one scale for all: a multiple of a quarter of it, at most 36 * 192 of them
        np.testing.assert_array_equal(_host(got), want.astype(np.float32))


def test_linear_takes_the_tensor_scales():
    a, w = _random(5, 64, "nv", 1), _random(70, 64, "nv", 2)
    want, _ = oracle_fp4.linear(oracle_fp4.values(*a, "nv", 0.25), oracle_fp4.values(*w, "nv", 2.0 ** -10), 3.0)
    got = binding.fp4_linear(_matrix(*a, "nv", 0.25), _matrix(*w, "nv", 2.0 ** -10), F32, alpha=3.0)
    # the sum is exact; times alpha it is rounded once
    assert (np.abs(_host(got) - want) <= np.abs(want) * 2.0 ** -24).all()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_linear_of_nan_blocks(fmt):
    """Rows with a NaN scale give NaN, the others what they give without it."""
    a, w = _random(9, 128, fmt, 1), _random(140, 128, fmt, 2)
    a[1][4, 2] = 255 if fmt == "mx" else 127
    w[1][130, 0] = 255 if fmt == "mx" else 127
    want, _ = oracle_fp4.linear(oracle_fp4.values(*a, fmt), oracle_fp4.values(*w, fmt))
    assert np.isnan(want[4]).all() and np.isnan(want[:, 130]).all() and np.isnan(want).sum() == 140 + 8
    got = binding.fp4_linear(_matrix(*a, fmt), _matrix(*w, fmt), F32)
    np.testing.assert_array_equal(_host(got), want.astype(np.float32))


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("R,V,K", [(1, 4096, 4096), (60, 1000, 2080), (300, 640, 1000)])
def test_quantize_then_linear(fmt, dtype, R, V, K):
    """Features and a weight as they come.  An fp32 sum of K terms, in any order and cut off instead
    of rounded, is off by at most K 2^-23 of the sum of their magnitudes; then one rounding."""
    g = torch.Generator(device=DEV).manual_seed(7)
    x = torch.randn((R, K), generator=g, device=DEV).to(BF)
    wt = (torch.randn((V, K), generator=g, device=DEV) * 0.02).to(BF)
    a, w = binding.fp4_quantize(x, fmt, TS[fmt]), binding.fp4_quantize(wt, fmt, 1.0 if fmt == "mx" else 2.0 ** -10)
    got = binding.fp4_linear(a, w, dtype)
    av, wv = (oracle_fp4.values(*oracle_fp4.unpack(m.codes.cpu().numpy(), m.scales.cpu().numpy(), m.rows, m.cols, fmt),
                                fmt, m.tensor_scale) for m in (a, w))
    want, size = oracle_fp4.linear(av, wv)
    tol = size * K * 2.0 ** -23 + np.abs(want) * torch.finfo(dtype).eps / 2 * 1.01
    assert (np.abs(_host(got) - want) <= tol).all()


def test_linear_repeats_bit_for_bit():
    a = binding.fp4_quantize(torch.randn((100, 4096), device=DEV).to(BF))
    w = binding.fp4_quantize(torch.randn((5000, 4096), device=DEV).to(BF))
    first = binding.fp4_linear(a, w, F32)
    for _ in range(3):
        assert torch.equal(first, binding.fp4_linear(a, w, F32))


def test_empty():
    q = binding.fp4_quantize(torch.empty((0, 64), dtype=BF, device=DEV))
    assert q.codes.shape == (0, 32) and binding.fp4_dequantize(q).shape == (0, 64)
    w = binding.fp4_quantize(torch.randn((4, 64), dtype=F32, device=DEV))
    assert binding.fp4_linear(q, w).shape == (0, 4)
