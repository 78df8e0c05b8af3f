"""The 8-bit operators from their definitions, in 64 bits (NumPy), for the tests."""
from __future__ import annotations

import numpy as np

TINY = 2.0 ** -100


def blocks(n: int) -> int:
    return (n + 127) // 128


def _e4m3_table() -> np.ndarray:
    """The non-negative e4m3 numbers in the order of their codes (0 .. 126)."""
    code = np.arange(127)
    e, m = code >> 3, code & 7
    return np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))


E4M3 = _e4m3_table()


def decode(codes: np.ndarray) -> np.ndarray:
    """Values of e4m3 code bytes."""
    c = codes.astype(np.int64)
    v = np.append(E4M3, np.nan)[c & 127]
    return np.where(c & 128, -v, v)


def round_e4m3(v: np.ndarray) -> np.ndarray:
    """The nearest e4m3 number to each value (ties to the even code; at most 448)."""
    a = np.abs(v)
    hi = np.clip(np.searchsorted(E4M3, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = E4M3[hi] - a, a - E4M3[lo]
    take_hi = (up < down) | ((up == down) & (hi % 2 == 0))
    return np.copysign(np.where(take_hi, E4M3[hi], E4M3[lo]), v)


def quantize(x: np.ndarray, block_rows: int = 1):
    """(values of the codes, scales) of a matrix [R][K]; the definition's fp32 steps one by one."""
    x = x.astype(np.float32)
    R, K = x.shape
    rb = -(-R // block_rows)
    m = np.zeros((rb * block_rows, blocks(K) * 128), np.float32)
    m[:R, :K] = np.abs(x)
    a = np.maximum(m.reshape(rb, block_rows, blocks(K), 128).max((1, 3)), np.float32(TINY))
    inv = np.float32(448) / a
    v = x * spread(inv, block_rows, R, K)
    assert v.dtype == np.float32
    return round_e4m3(v.astype(np.float64)), (a / np.float32(448)).astype(np.float32)


def spread(scales: np.ndarray, block_rows: int, R: int, K: int) -> np.ndarray:
    return np.repeat(np.repeat(scales, block_rows, 0)[:R], 128, 1)[:, :K]


def values(codes: np.ndarray, scales: np.ndarray, block_rows: int) -> np.ndarray:
    """What codes (their values) and scales stand for, in 64 bits."""
    return codes.astype(np.float64) * spread(scales.astype(np.float64), block_rows, *codes.shape)


def product_bound(av: np.ndarray, bv: np.ndarray) -> np.ndarray:
    """How far a computed a b^T may be from the exact one, before its last rounding.

    The products of two codes are exact.  A sum of n terms in fp32 is off by at
    most n units of 2^-23 of the sum of magnitudes, whether an addition rounds
    or truncates: 128 terms of a block, then one product of scales, one by the
    scale and one addition for each block.
    """
    return (128 + 3 * blocks(av.shape[1]) + 8) * 2.0 ** -23 * (np.abs(av) @ np.abs(bv).T)
