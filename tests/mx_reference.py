"""Plain 64-bit restatement of the microscaled (MX) operators for the tests:
numpy, value by value from the format's definition, no code of the library.

A block of 32 values has the scale 2^(floor(log2 max|v|) - emax), not below
2^-127, and codes round(v / scale) to nearest even, cut at the largest code;
a block with an infinity or a NaN has scale byte 255 and zero codes."""
from __future__ import annotations

import numpy as np

EMAX = {4: 2, 8: 8}


def code_values(bits: int) -> np.ndarray:
    """The value of every code, from its fields: sign, exponent, mantissa."""
    n, ebits, mbits, bias = (16, 2, 1, 1) if bits == 4 else (256, 4, 3, 7)
    out = np.empty(n)
    for c in range(n):
        sign = -1.0 if c >= n // 2 else 1.0
        e, m = (c >> mbits) & ((1 << ebits) - 1), c & ((1 << mbits) - 1)
        if bits == 8 and e == 15 and m == 7:
            out[c] = np.nan
        elif e == 0:
            out[c] = sign * m * 2.0 ** (1 - bias - mbits)
        else:
            out[c] = sign * (1 + m * 2.0 ** -mbits) * 2.0 ** (e - bias)
    return out


def nearest_code(u: np.ndarray, bits: int) -> np.ndarray:
    """The code of each scaled value, sign included (also of a zero)."""
    half = 8 if bits == 4 else 127      # non-negative finite codes 0 .. half - 1
    grid = code_values(bits)[:half]
    a = np.minimum(np.abs(u), grid[-1])
    hi = np.searchsorted(grid, a)        # grid[hi-1] < a <= grid[hi]
    lo = np.maximum(hi - 1, 0)
    up, down = grid[hi] - a, a - grid[lo]
    c = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (c + np.where(np.signbit(u), 1 << (bits - 1), 0)).astype(np.uint8)


def padded(K: int) -> int:
    return -(-K // 128) * 128


def blocks(v: np.ndarray) -> np.ndarray:
    rows, K = v.shape
    b = np.zeros((rows, padded(K)))
    b[:, :K] = v
    return b.reshape(rows, -1, 32)


def scale_bytes(v: np.ndarray, bits: int) -> np.ndarray:
    """[rows, Kp/32]"""
    top = np.abs(blocks(v)).max(-1)
    bad = ~np.isfinite(top)
    _, e = np.frexp(np.where(bad | (top == 0), 1.0, top))   # top = f·2^e, 1/2 <= f < 1
    byte = np.clip(e - 1 - EMAX[bits] + 127, 0, 254)
    byte = np.where(top == 0, 0, byte)
    return np.where(bad, 255, byte).astype(np.uint8)


def codes_under(v: np.ndarray, byte: np.ndarray, bits: int) -> np.ndarray:
    """Codes [rows, Kp] of v under given scale bytes (zero where the byte is 255)."""
    b = blocks(v)
    ok = byte != 255
    with np.errstate(over="ignore"):
        u = np.where(ok[..., None], b, 0.0) * np.exp2(127.0 - byte.astype(np.float64))[..., None]
    return np.where(ok[..., None], nearest_code(u, bits), 0).reshape(v.shape[0], -1).astype(np.uint8)


def quantize(v: np.ndarray, bits: int):
    byte = scale_bytes(v, bits)
    return codes_under(v, byte, bits), byte


def pack(codes: np.ndarray, bits: int) -> np.ndarray:
    return codes if bits == 8 else codes[:, 0::2] | (codes[:, 1::2] << 4)


def unpack(packed: np.ndarray, bits: int) -> np.ndarray:
    if bits == 8:
        return packed
    out = np.empty((packed.shape[0], 2 * packed.shape[1]), np.uint8)
    out[:, 0::2], out[:, 1::2] = packed & 15, packed >> 4
    return out


def tile(byte: np.ndarray) -> np.ndarray:
    """Scale bytes [rows, Kp/32] in tiles [ceil(rows/128), Kp/128, 512], entry by entry."""
    rows, nb = byte.shape
    out = np.zeros((-(-rows // 128), nb // 4, 512), np.uint8)
    for r in range(rows):
        for j in range(4):
            out[r // 128, :, 16 * (r % 32) + 4 * (r % 128 // 32) + j] = byte[r, j::4]
    return out


def untile(tiles: np.ndarray, rows: int) -> np.ndarray:
    out = np.empty((rows, tiles.shape[1] * 4), np.uint8)
    for r in range(rows):
        for j in range(4):
            out[r, j::4] = tiles[r // 128, :, 16 * (r % 32) + 4 * (r % 128 // 32) + j]
    return out


def values(codes: np.ndarray, byte: np.ndarray, bits: int) -> np.ndarray:
    """What unpacked codes [rows, Kp] and scale bytes stand for."""
    s = np.where(byte == 255, np.nan, np.exp2(byte.astype(np.float64) - 127))
    return code_values(bits)[codes] * np.repeat(s, 32, axis=1)


def rmsnorm(x: np.ndarray, weight: np.ndarray, eps: float, residual: np.ndarray | None = None):
    """(v, h)"""
    h = x if residual is None else x + residual
    return h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * weight, h


def swiglu(gate: np.ndarray, up: np.ndarray) -> np.ndarray:
    with np.errstate(over="ignore"):
        return gate / (1 + np.exp(-gate)) * up
