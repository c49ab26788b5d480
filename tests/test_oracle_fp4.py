"""Pins of the 4-bit oracle: blocks worked by hand, the formats' number lists, brute force over the grid, the
layout against an independent walk through memory."""
import numpy as np
import pytest

from oracle import fp4


def test_number_lists():
    e4m3 = fp4.e4m3_values()
    assert e4m3[0] == 0 and e4m3[1] == 2.0 ** -9 and e4m3[7] == 7 * 2.0 ** -9  # subnormal
    assert e4m3[8] == 2.0 ** -6 and e4m3[0x38] == 1.0 and e4m3[0x7e] == 448.0
    assert (np.diff(e4m3) > 0).all()
    # e2m1: two exponent bits (bias 1) and one of the significand
    for code in range(8):
        e, m = code >> 1, code & 1
        assert fp4.GRID[code] == (m / 2 if e == 0 else (1 + m / 2) * 2.0 ** (e - 1))


def test_mx_block_by_hand():
    x = np.zeros((1, 40), dtype=np.float32)
    x[0, :8] = [7.9, -4.0, 0.25, 0.26, 0.75, 1.25, -2.5, 3.5]  # floor(log2 7.9) - 2 = 0: scale 1
    x[0, 32:36] = [96.0, 80.0, -17.0, 8.0]  # floor(log2 96) - 2 = 4: scale 16
    codes, scales = fp4.quantize(x, "mx")
    assert scales.tolist() == [[127, 131]]
    v = fp4.values(codes, scales, "mx")[0]
    assert v[:8].tolist() == [6, -4, 0, 0.5, 1, 1, -2, 4]
    assert v[32:36].tolist() == [96, 64, -16, 8]  # 80 / 16 = 5 lies between 4 and 6: the even code, 4


def test_nv_block_by_hand():
    x = np.zeros((1, 17), dtype=np.float32)
    x[0, :4] = [9.0, -3.0, 0.375, 0.38]  # 9 / 6 = 1.5
    x[0, 16] = 0.1  # 0.1 / 6 = 0.016667 lies between the e4m3 numbers 8 / 512 and 9 / 512 = 0.017578
    codes, scales = fp4.quantize(x, "nv")
    assert fp4.e4m3_values()[scales[0]].tolist() == [1.5, 9 / 512]
    v = fp4.values(codes, scales, "nv")[0]
    assert v[:4].tolist() == [9, -3, 0, 0.75] and v[16] == 6 * 9 / 512
    # the tensor scale moves the block scales, not the values
    c2, s2 = fp4.quantize(x, "nv", 0.25)
    assert fp4.e4m3_values()[s2[0]].tolist() == [6.0, 9 / 128] and (fp4.values(c2, s2, "nv", 0.25)[0] == v).all()


def test_special_blocks():
    x = np.ones((1, 96), dtype=np.float32)
    x[0, :32] = 0
    x[0, 40] = np.inf
    x[0, 64] = np.nan
    codes, scales = fp4.quantize(x, "mx")
    assert scales.tolist() == [[0, 255, 255]] and not codes.any()
    v = fp4.values(codes, scales, "mx")
    assert (v[0, :32] == 0).all() and np.isnan(v[0, 32:]).all()
    codes, scales = fp4.quantize(x, "nv")
    assert scales.tolist() == [[0, 0, 127, 35, 127, 35]]  # 1 / 6: 11 / 64
    # the largest and the smallest scales
    big = np.full((1, 16), 3e38, dtype=np.float32)
    assert fp4.quantize(big, "nv")[1][0, 0] == 126 and fp4.quantize(big, "mx")[1][0, 0] == 127 + 125
    tiny = np.full((1, 16), 1e-45, dtype=np.float32)
    assert fp4.quantize(tiny, "nv")[1][0, 0] == 0 and fp4.quantize(tiny, "mx")[1][0, 0] == 0


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_every_code_is_the_nearest(fmt):
    rng = np.random.default_rng(4)
    x = (rng.standard_normal((6, 70)) * 2.0 ** rng.integers(-6, 6, (6, 1))).astype(np.float32)
    codes, scales = fp4.quantize(x, fmt)
    v = fp4.values(codes, scales, fmt)
    n = fp4.BLOCK[fmt]
    for r in range(6):
        for i in range(70):
            s = fp4.scale_value(scales[r, i // n], fmt)
            best = min(abs(x[r, i] - g * s * sign) for g in fp4.GRID for sign in (1, -1))
            assert abs(x[r, i] - v[r, i]) == best


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("R,K", [(1, 1), (3, 33), (130, 150), (300, 64)])
def test_layout(fmt, R, K):
    rng = np.random.default_rng(R)
    blocks = -(-K // fp4.BLOCK[fmt])
    codes = rng.integers(0, 16, (R, K)).astype(np.uint8)
    scales = rng.integers(1, 127, (R, blocks)).astype(np.uint8)
    packed, tiled = fp4.pack(codes, scales, fmt)
    assert packed.shape == (R, 16 * (-(-K // 32)))
    assert tiled.size == -(-R // 128) * (-(-blocks // 4)) * 512
    back = fp4.unpack(packed, tiled, R, K, fmt)
    assert (back[0] == codes).all() and (back[1] == scales).all()
    # the same memory as one array of tiles [row tile, group, r % 32, r / 32 % 4, b % 4]
    five = tiled.reshape(-(-R // 128), -1, 32, 4, 4).transpose(0, 3, 2, 1, 4).reshape(-(-R // 128) * 128, -1)
    assert (five[:R, :blocks] == scales).all()
    assert five.sum() == scales.sum()  # padding is zero
    assert sum(int(p & 15) + int(p >> 4) for p in packed.reshape(-1)) == int(codes.sum())


def test_linear():
    a, w = np.array([[1.0, 2, -3]]), np.array([[1.0, 1, 1], [0.5, 0, 2]])
    out, size = fp4.linear(a, w, 2.0)
    assert out.tolist() == [[0.0, -11.0]] and size.tolist() == [[12.0, 13.0]]
