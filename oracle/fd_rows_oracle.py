"""fp64 oracle of the cache-row operations: head norm, rotation, 4-bit blocks.

TEST INFRASTRUCTURE ONLY, like the decode oracle: plain numpy arrays in and out, no code
shared with the CUDA path.  Every function is pinned by ``tests/test_oracle_rows.py``.
"""
from __future__ import annotations

import numpy as np

from .fd_oracle import widen

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# The finite non-negative values of E4M3, in code order.
E4M3 = widen(np.arange(127, dtype=np.uint8), "e4m3")


def nearest_code(a, grid):
    """Index of the value of `grid` nearest to each a >= 0: ties to even, saturating."""
    a = np.asarray(a, dtype=np.float64)
    hi = np.searchsorted(grid, a).clip(1, len(grid) - 1)
    lo = hi - 1
    down, up = a - grid[lo], grid[hi] - a
    take_lo = (down < up) | ((down == up) & (lo % 2 == 0))
    return np.where(a >= grid[-1], len(grid) - 1, np.where(take_lo, lo, hi))


def quantise(x):
    """Codes [..., n] (sign in bit 3) and E4M3 scale bytes [..., n / 16] of x (finite)."""
    x = np.asarray(x, dtype=np.float64)
    y = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    amax = np.abs(y).max(-1)
    # The scale is the E4M3 rounding of an fp32 quotient.
    scale = nearest_code((amax.astype(np.float32) / np.float32(6)).astype(np.float64), E4M3)
    s = E4M3[scale][..., None]
    mag = np.divide(np.abs(y), s, out=np.zeros_like(y), where=s > 0)
    code = nearest_code(mag, E2M1) + 8 * np.signbit(y)
    return code.reshape(x.shape).astype(np.uint8), scale.astype(np.uint8)


def dequantise(codes, scales):
    """Values of codes and scale bytes (a NaN scale makes its 16 values NaN)."""
    mag = E2M1[codes & 7]
    v = np.where(codes & 8, -mag, mag).reshape(*codes.shape[:-1], codes.shape[-1] // 16, 16)
    return (v * widen(scales, "e4m3")[..., None]).reshape(codes.shape)


def _offsets(which, d):
    """Byte of every (row, element) pair's code in a block, and of its scale."""
    r, e = np.meshgrid(np.arange(16), np.arange(d), indexing="ij")
    if which == "k":
        return r * (d // 2) + e // 2, 8 * d + r * (d // 16) + e // 16
    g = e // (d // 8)
    swap = 4 * ((g if d == 128 else g // 2) % 2)
    byte = g * d + ((r // 2) ^ swap) * (d // 8) + (r % 2) * (d // 16) + (e % (d // 8)) // 2
    return byte, 8 * d + 16 * (e // 16) + r


def unpack_blocks(pool, which):
    """Codes and scale bytes [tokens, Hkv, d], [tokens, Hkv, d / 16] of blocks [n, Hkv, 9 d]."""
    n, H, size = pool.shape
    d = size // 9
    byte, scale = _offsets(which, d)
    odd = (np.arange(d) % 2).astype(bool)
    raw = pool[:, :, byte]                                    # [n, H, 16, d]
    codes = np.where(odd, raw >> 4, raw & 15)
    scales = pool[:, :, scale[:, ::16]]
    to = lambda x: x.transpose(0, 2, 1, 3).reshape(16 * n, H, -1)  # noqa: E731
    return to(codes), to(scales)


def pack_blocks(codes, scales, which):
    """Inverse of unpack_blocks; the number of tokens is a multiple of 16."""
    tokens, H, d = codes.shape
    byte, scale = _offsets(which, d)
    pool = np.zeros((tokens // 16, H, 9 * d), dtype=np.uint8)
    c = codes.reshape(-1, 16, H, d).transpose(0, 2, 1, 3)
    pool[:, :, byte[:, 0::2]] = c[..., 0::2] | (c[..., 1::2] << 4)
    pool[:, :, scale[:, ::16]] = scales.reshape(-1, 16, H, d // 16).transpose(0, 2, 1, 3)
    return pool


def norm_rotate(x, weight=None, offset=0.0, eps=1e-6, norm=False, inv_freq=(), axes=None,
                positions=None, interleaved=False, scale=1.0):
    """x [T, H, d] float64: RMS norm of each head (if `norm`), then the rotation of its first
    2 len(inv_freq) elements by positions [axes, T] x inv_freq."""
    y = np.array(x, dtype=np.float64)
    if norm:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps)
        if weight is not None:
            y = y * (np.asarray(weight, dtype=np.float64) + offset)
    n = len(inv_freq)
    axes = [0] * n if axes is None else axes
    out = y.copy()
    for i in range(n):
        th = np.asarray(positions)[axes[i]].astype(np.float64) * inv_freq[i]
        c, s = scale * np.cos(th)[:, None], scale * np.sin(th)[:, None]
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        out[..., ia] = y[..., ia] * c - y[..., ib] * s
        out[..., ib] = y[..., ia] * s + y[..., ib] * c
    return out, y
