"""CPU oracle of 8-bit matrices with a power of two for each block of 128 (test
infrastructure only).

Plain NumPy in fp64, from tables of the formats' values, sharing no code with the
HIP library.
"""
from __future__ import annotations

import numpy as np

FORMATS = {"e4m3": (4, 3, 7, 448.0), "e5m2": (5, 2, 15, 57344.0)}   # exponent, mantissa bits, bias, largest


def decode(codes: np.ndarray, fmt: str) -> np.ndarray:
    """The value of each code: E4M3 has no infinity and one NaN a sign (S.1111.111),
    E5M2 those of IEEE 754."""
    ebits, mbits, bias, _ = FORMATS[fmt]
    c = np.asarray(codes, dtype=np.uint8).astype(np.int64)
    e, m = c >> mbits & (1 << ebits) - 1, c & (1 << mbits) - 1
    v = np.where(e == 0, m * 2.0 ** (1 - bias - mbits), (1 + m / 2.0 ** mbits) * 2.0 ** (e - bias))
    if fmt == "e4m3":
        v = np.where((e == 15) & (m == 7), np.nan, v)
    else:
        v = np.where(e == 31, np.where(m == 0, np.inf, np.nan), v)
    return np.where(c & 128, -v, v)


def _tables(fmt: str):
    """The non-negative finite values in order, code by code."""
    v = decode(np.arange(128), fmt)
    return v[np.isfinite(v)]


def encode(x: np.ndarray, fmt: str, saturate: bool = False) -> np.ndarray:
    """The code nearest to x, ties to the even code; what is not finite as the module
    says.  |x| is at most the largest value, unless saturate takes it there."""
    x = np.asarray(x, dtype=np.float64)
    v = _tables(fmt)
    a = np.abs(np.where(np.isfinite(x), x, 0.0))
    if saturate:
        a = np.minimum(a, v[-1])
    assert (a <= v[-1]).all()
    hi = np.searchsorted(v, a)                  # v[hi - 1] < a <= v[hi]
    lo = np.maximum(hi - 1, 0)
    up = v[hi] - a < a - v[lo]
    tie = v[hi] - a == a - v[lo]
    code = np.where(up | (tie & (hi % 2 == 0)), hi, lo)
    code = np.where(a == v[hi], hi, code)
    nan = 0x7F
    if fmt == "e5m2":
        code = np.where(np.isinf(x), 0x7C, code)
        code = np.where(np.isnan(x), nan, code)
    else:
        code = np.where(~np.isfinite(x), nan, code)
    return (code + np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def scale_byte(a: np.ndarray, fmt: str) -> np.ndarray:
    """The smallest byte with a <= fmax 2^(byte - 127)."""
    top = FORMATS[fmt][3] * 2.0 ** (np.arange(256.0) - 127)
    return np.searchsorted(top, np.asarray(a, dtype=np.float64)).astype(np.uint8)


def _sides(blocks: str):
    return {"rows": (1, 128), "cols": (128, 1), "tiles": (128, 128)}[blocks]


def _spread(per_block: np.ndarray, blocks: str, rows: int, cols: int) -> np.ndarray:
    """A value for each block to one for each element."""
    r, c = _sides(blocks)
    return np.repeat(np.repeat(per_block, r, 0)[:rows], c, 1)[:, :cols]


def block_bytes(x: np.ndarray, blocks: str, fmt: str, top: int = 0) -> np.ndarray:
    """[block rows, block columns] of x, whose first row lies `top` rows into a block."""
    r, c = _sides(blocks)
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(np.where(np.isfinite(x), x, 0.0))
    down, across = -(-(top + x.shape[0]) // r), -(-x.shape[1] // c)
    full = np.zeros((down * r, across * c))
    full[top:top + x.shape[0], :x.shape[1]] = a
    return scale_byte(full.reshape(down, r, across, c).max((1, 3)), fmt)


def quantize(x: np.ndarray, blocks: str, fmt: str):
    """(codes, bytes), bytes laid out as the library does: a line of them for each 128
    columns of "rows", for each 128 rows otherwise."""
    b = block_bytes(x, blocks, fmt)
    s = 2.0 ** (_spread(b, blocks, *x.shape).astype(np.float64) - 127)
    return encode(np.asarray(x, dtype=np.float64) / s, fmt), b.T.copy() if blocks == "rows" else b


def values(codes: np.ndarray, lines: np.ndarray, blocks: str, fmt: str) -> np.ndarray:
    """What codes stand for, in fp64 (byte 255: NaN)."""
    v = decode(codes, fmt)
    if blocks == "tensor":
        return v
    b = lines.T if blocks == "rows" else lines
    s = np.where(b == 255, np.nan, 2.0 ** (b.astype(np.float64) - 127))
    return v * _spread(s, blocks, *codes.shape)


def product_tolerance(a: np.ndarray, b: np.ndarray, c: np.ndarray) -> np.ndarray:
    """How far a bf16 result may be from c = a b in fp64.

    Of eight neighbouring products each loses less than 2^-13 of the power of two of
    the largest, seven at most lose any: 7 2^-13 of the sum of magnitudes S.  An element
    of the result takes part in fewer than K / 8 + K / 128 + 24 fp32 additions, each off
    by half of 2^-23 of at most S.  Then the rounding to bf16, 2^-8 of the result."""
    k = a.shape[1]
    s = np.abs(a) @ np.abs(b)
    off = s * (7 * 2.0 ** -13 + (k / 8 + k / 128 + 24) * 2.0 ** -24)
    return 2.0 ** -8 * np.abs(c) + (1 + 2.0 ** -8) * off + 2.0 ** -133
