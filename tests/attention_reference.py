"""Plain 64-bit restatement of the attention operators for the tests: numpy,
from the definitions, no code of the library.  A cache is a dict of uint8
arrays k_codes, v_codes [pages, kv heads, page, D·bits/8] and k_scales,
v_scales [pages, kv heads, page, 4]; a batch is (starts, lengths, table)."""
from __future__ import annotations

import numpy as np

import mx_reference as mx


def turned(x: np.ndarray, positions, frequencies, interleaved: bool = False, magnitude: float = 1.0) -> np.ndarray:
    """x [T, H, D] with its first pairs turned, pair by pair; angles in extended precision where there is one."""
    out = np.array(x, np.float64)
    n = len(frequencies)
    p = np.asarray(positions).astype(np.longdouble)
    for i, f in enumerate(np.asarray(frequencies, np.float64)):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        angle = np.fmod(p * np.longdouble(f), 2 * np.arctan2(np.longdouble(0), np.longdouble(-1)))
        c = magnitude * np.cos(angle).astype(np.float64)[:, None]
        s = magnitude * np.sin(angle).astype(np.float64)[:, None]
        out[..., a] = x[..., a] * c - x[..., b] * s
        out[..., b] = x[..., b] * c + x[..., a] * s
    return out


def places(batch, page: int):
    """Of each row of the batch: (row, sequence, position, page number, place), rows at negative positions left out."""
    starts, lengths, table = (np.asarray(a) for a in batch)
    for i in range(len(lengths)):
        for t in range(starts[i], starts[i + 1]):
            p = int(lengths[i]) - int(starts[i + 1]) + t
            if p >= 0:
                yield t, i, p, int(table[i][p // page]), p % page


def head_codes(v: np.ndarray, bits: int):
    """Packed codes and scale bytes [4] of one head's values."""
    codes, byte = mx.quantize(v[None], bits)
    return mx.pack(codes, bits)[0][:len(v) * bits // 8], np.concatenate([byte[0][:len(v) // 32], np.zeros(4, np.uint8)])[:4]


def head_values(codes: np.ndarray, scales: np.ndarray, bits: int) -> np.ndarray:
    """[..., D] values of packed codes [..., D·bits/8] under scale bytes [..., 4]."""
    c = mx.unpack(codes.reshape(-1, codes.shape[-1]), bits)
    byte = scales.reshape(-1, 4)[:, :c.shape[1] // 32]
    return mx.values(c, byte, bits).reshape(*codes.shape[:-1], -1)


def cached(cache, what: str, batch, i: int, bits: int) -> np.ndarray:
    """[lengths[i], kv heads, D]: all of what sequence i has in the cache."""
    _, lengths, table = batch
    page = cache[what + "_codes"].shape[2]
    n = int(lengths[i])
    pages = [int(table[i][p]) for p in range(-(-n // page))]
    v = [head_values(cache[what + "_codes"][p], cache[what + "_scales"][p], bits).transpose(1, 0, 2) for p in pages]
    return np.concatenate(v)[:n] if v else np.zeros((0, cache[what + "_codes"].shape[1], 0))


def attention(q: np.ndarray, cache, batch, bits: int, scale: float, causal: bool = True):
    """y [T, H, D], and what its error scales with: Σ P|v|, the largest scale·Σ|q k|, the largest P·max|v| and the
    number of keys, each broadcast to y.  Rows of no sequence are NaN in y."""
    starts, lengths, _ = batch
    T, H, D = q.shape
    y = np.full(q.shape, np.nan)
    spread, size, most, keys = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape)
    for i in range(len(lengths)):
        k, v = (cached(cache, w, batch, i, bits) for w in "kv")
        n = int(starts[i + 1]) - int(starts[i])
        for t in range(n):
            sees = max(0, int(lengths[i]) - n + t + 1 if causal else int(lengths[i]))
            for h in range(H):
                row, g = int(starts[i]) + t, h // (H // max(1, cache["k_codes"].shape[1]))
                if sees == 0:
                    y[row, h] = 0
                    continue
                with np.errstate(invalid="ignore"):
                    s = scale * (k[:sees, g] @ q[row, h])
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    y[row, h] = p @ v[:sees, g]
                spread[row, h] = p @ np.abs(v[:sees, g])
                size[row, h] = scale * (np.abs(k[:sees, g]) @ np.abs(q[row, h])).max()
                most[row, h] = np.nanmax(np.append(p * np.nanmax(np.abs(v[:sees, g]), -1), 0))
                keys[row, h] = sees
    return y, spread, size, most, keys
