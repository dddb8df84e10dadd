"""The rotating cache write's rule in numpy binary32, a step at a time as the
entry points state it, for comparing bytes."""
from __future__ import annotations

import numpy as np
import torch

F = np.float32


def turned(x, table, positions, axis, interleaved):
    """x [T, heads, D] float32, table [max_position, R], positions [axes, T], axis [R / 2]: float32, every
    product and sum rounded by itself."""
    x = x.copy()
    R = table.shape[1]
    pos = np.asarray(positions)[np.asarray(axis)].T                      # [T, R / 2]
    pair = np.arange(R // 2)
    c, s = table[pos, pair][:, None], table[pos, R // 2 + pair][:, None]
    a = x[..., 0:R:2].copy() if interleaved else x[..., :R // 2].copy()
    b = x[..., 1:R:2].copy() if interleaved else x[..., R // 2:R].copy()
    assert a.dtype == b.dtype == c.dtype == F
    new_a, new_b = a * c - b * s, b * c + a * s
    if interleaved:
        x[..., 0:R:2], x[..., 1:R:2] = new_a, new_b
    else:
        x[..., :R // 2], x[..., R // 2:R] = new_a, new_b
    return x


def e4m3_rows(x, scale):
    """float32 rows as bytes of e4m3 codes."""
    y = torch.from_numpy((x / F(scale)).clip(F(-448), F(448)))
    return y.to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def q4_rows(x):
    """float32 rows [..., D] as q4_0 bytes [..., 9 D / 16]."""
    blocks = x.reshape(*x.shape[:-1], -1, 32)
    at = np.abs(blocks).argmax(-1)                                       # the first of the largest
    m = np.take_along_axis(blocks, at[..., None], -1)
    d = m / F(-8)
    inv = np.where(d != 0, F(1) / np.where(d != 0, d, F(1)), F(0)).astype(F)
    y = blocks * inv + F(8.5)
    code = np.where(y >= 15, 15, np.where(y >= 0, np.trunc(y), 0)).astype(np.uint8)
    code = code[..., :16] | (code[..., 16:] << 4)
    with np.errstate(over="ignore"):
        scales = np.ascontiguousarray(d[..., 0].astype(np.float16)).view(np.uint8)
    return np.concatenate([scales, code.reshape(*x.shape[:-1], -1)], -1)


def q4_values(rows):
    """The float64 values that q4_0 rows stand for."""
    n = rows.shape[-1] // 9
    d = np.ascontiguousarray(rows[..., :n]).view(np.float16).astype(np.float64)
    code = rows[..., n:].reshape(*rows.shape[:-1], n // 2, 16)
    code = np.concatenate([code & 15, code >> 4], -1).astype(np.float64) - 8
    return (code * d[..., None]).reshape(*rows.shape[:-1], 16 * n)
