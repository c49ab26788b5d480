"""Oracle of block-scaled 4-bit floating point: TEST INFRASTRUCTURE ONLY (tests and smoke may use it; the
CUDA library never does).  Codes are the indices of GRID with the sign in bit 3, scales bytes.

Readings taken here:
  - "mx" (OCP Microscaling Formats specification 1.0, MXFP4): blocks of 32 along a row, scale
    2^(floor(log2 m) - 2) for the largest magnitude m (2 is the exponent of the largest e2m1 number),
    clamped to 2^-127 .. 2^127, 2^-127 for m = 0; byte e + 127;
  - "nv": blocks of 16, scale s * tensor_scale, s the e4m3 number nearest to m / (6 tensor_scale), halves to
    the even code, at most 448;
  - a code is the grid value nearest to |x| / scale, halves to the even code, beyond 6: 6; a block
    whose scale is 0 has codes 0;
  - a block that holds NaN or an infinity has the scale that stands for NaN (255; 127) and codes 0.
Everything is compared exactly: |x| with midpoint * scale, both numbers of few bits, in 64 bits.
"""
import numpy as np

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
BLOCK = {"mx": 32, "nv": 16}


def bf16(x):
    """float32 values of raw bf16 bits (uint16)."""
    return (np.asarray(x, dtype=np.uint16).astype(np.uint32) << 16).view(np.float32)


def e4m3_values():
    """The 127 non-negative finite e4m3 numbers, by code."""
    v = []
    for c in range(127):
        e, m = c >> 3, c & 7
        v.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return np.array(v)


def _nearest(value, grid, unit):
    """Code of the grid value nearest to value / unit, halves to the even code."""
    code = 0
    for i in range(1, len(grid)):
        mid = (grid[i - 1] + grid[i]) / 2 * unit
        if value > mid or (value == mid and i % 2 == 0):
            code = i
    return code


def scale_value(byte, fmt, tensor_scale=1.0):
    if fmt == "mx":
        return np.nan if byte == 255 else 2.0 ** (int(byte) - 127)
    return np.nan if byte == 127 else e4m3_values()[byte] * tensor_scale


def quantize(x, fmt, tensor_scale=1.0):
    """x [R, K] (float32 values).  Returns codes [R, K] uint8 and scale bytes [R, blocks] uint8."""
    x = np.asarray(x, dtype=np.float64)
    R, K = x.shape
    n = BLOCK[fmt]
    blocks = -(-K // n)
    codes = np.zeros((R, K), dtype=np.uint8)
    scales = np.zeros((R, blocks), dtype=np.uint8)
    grid8 = e4m3_values()
    for r in range(R):
        for b in range(blocks):
            v = x[r, b * n:(b + 1) * n]
            if not np.isfinite(v).all():
                scales[r, b] = 255 if fmt == "mx" else 127
                continue
            m = np.abs(v).max()
            if fmt == "mx":
                e = -127
                while e < 127 and 2.0 ** (e + 1) * 4 <= m:
                    e += 1
                scales[r, b] = e + 127
            else:  # m / (6 ts) against the midpoints of the e4m3 numbers
                i = int(np.searchsorted(grid8 * (6 * tensor_scale), m, side="right")) - 1
                if i < 126:
                    mid = (grid8[i] + grid8[i + 1]) / 2 * (6 * tensor_scale)
                    if m > mid or (m == mid and i % 2 == 1):
                        i += 1
                scales[r, b] = i
            s = scale_value(scales[r, b], fmt, tensor_scale)
            if s == 0:
                continue
            for j, y in enumerate(v):
                codes[r, b * n + j] = _nearest(abs(y), GRID, s) | (8 if np.signbit(y) else 0)
    return codes, scales


def values(codes, scales, fmt, tensor_scale=1.0):
    """[R, K] float64 of codes [R, K] and scale bytes [R, blocks]."""
    codes = np.asarray(codes)
    table = np.array([scale_value(b, fmt, tensor_scale) if (fmt == "mx" or b < 128) else np.nan
                      for b in range(256)])
    s = np.repeat(table[np.asarray(scales)], BLOCK[fmt], axis=1)[:, :codes.shape[1]]
    return GRID[codes & 7] * np.where(codes & 8, -1.0, 1.0) * s


def pack(codes, scales, fmt):
    """The memory of codes and scales, byte by byte from the layout's formulas."""
    R, K = codes.shape
    row = 16 * (-(-K // 32))
    out = np.zeros((R, row), dtype=np.uint8)
    for i in range(K):
        out[:, i // 2] |= (codes[:, i] << (4 * (i % 2))).astype(np.uint8)
    blocks = scales.shape[1]
    groups = -(-blocks // 4)
    s = np.zeros(-(-R // 128) * groups * 512, dtype=np.uint8)
    for r in range(R):
        for b in range(blocks):
            s[512 * ((r // 128) * groups + b // 4) + 16 * (r % 32) + 4 * (r // 32 % 4) + b % 4] = scales[r, b]
    return out, s


def unpack(packed, tiled, R, K, fmt):
    """pack's inverse: codes [R, K], scale bytes [R, blocks]."""
    packed, tiled = np.asarray(packed).reshape(R, -1), np.asarray(tiled).reshape(-1)
    codes = np.stack([(packed[:, i // 2] >> (4 * (i % 2))) & 15 for i in range(K)], axis=1)
    blocks = -(-K // BLOCK[fmt])
    groups = -(-blocks // 4)
    r, b = np.meshgrid(np.arange(R), np.arange(blocks), indexing="ij")
    at = 512 * ((r // 128) * groups + b // 4) + 16 * (r % 32) + 4 * (r // 32 % 4) + b % 4
    return codes, tiled[at]


def linear(a, w, alpha=1.0):
    """alpha * a w^T in 64 bits, and the sum of the products' magnitudes."""
    a, w = np.asarray(a, dtype=np.float64), np.asarray(w, dtype=np.float64)
    return alpha * (a @ w.T), abs(alpha) * (np.abs(a) @ np.abs(w).T)
