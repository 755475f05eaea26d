"""Pins of the cache-row oracle: hand-computed values and library routines (CPU only)."""
import numpy as np
import pytest

import oracle
from oracle import fd_rows_oracle as ro


def test_nearest_code_ties_to_even_and_saturates():
    a = [0.0, 0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.01, 6.0, 100.0, np.inf]
    assert oracle.nearest_code(a, ro.E2M1).tolist() == [0, 0, 1, 2, 2, 4, 4, 6, 6, 7, 7, 7, 7]


def test_e4m3_grid_matches_torch():
    import torch
    x = torch.linspace(0, 460, 20011).clamp(max=448)
    want = x.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(oracle.nearest_code(x.numpy(), ro.E4M3), want)


def test_quantise_by_hand():
    x = np.zeros((1, 32))
    x[0, :4] = [6.0, -3.0, 2.5, 0.25]       # scale 1: codes 7, 3|8 = 13, 2.5 -> 2 (code 4), 0
    x[0, 16:18] = [-12.0, 7.0]              # scale 2: codes 7|8, 3.5 -> 4 (code 6)
    codes, scales = oracle.quantise(x)
    assert codes[0, :4].tolist() == [7, 13, 4, 0] and codes[0, 16:18].tolist() == [15, 6]
    assert oracle.widen(scales, "e4m3").tolist() == [[1.0, 2.0]]
    y = oracle.dequantise(codes, scales)
    assert y[0, :4].tolist() == [6.0, -3.0, 2.0, 0.0] and y[0, 16:18].tolist() == [-12.0, 8.0]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("which", ["k", "v"])
def test_blocks_round_trip_and_fill_every_byte(d, which):
    rs = np.random.default_rng(d)
    codes = rs.integers(0, 16, (48, 3, d)).astype(np.uint8)
    scales = rs.integers(0, 256, (48, 3, d // 16)).astype(np.uint8)
    pool = oracle.pack_blocks(codes, scales, which)
    assert pool.shape == (3, 3, 9 * d)
    c, s = oracle.unpack_blocks(pool, which)
    assert np.array_equal(c, codes) and np.array_equal(s, scales)
    # One block of all-ones codes and scales leaves no byte unwritten.
    full = oracle.pack_blocks(np.full((16, 1, d), 15, np.uint8), np.full((16, 1, d // 16), 255, np.uint8), which)
    assert (full == 255).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rotate_closed_forms(interleaved):
    x = np.random.default_rng(1).standard_normal((3, 2, 64))
    n, _ = oracle.norm_rotate(x, norm=True, eps=0.0)
    assert np.allclose((n * n).mean(-1), 1.0)
    # A quarter turn of one pair; the others stay (frequency 0).
    freq = [np.pi / 2] + [0.0] * 15
    y, _ = oracle.norm_rotate(x, inv_freq=freq, positions=np.ones((1, 3)), interleaved=interleaved)
    a, b = (0, 1) if interleaved else (0, 16)
    assert np.allclose(y[..., a], -x[..., b]) and np.allclose(y[..., b], x[..., a])
    keep = [i for i in range(64) if i not in (a, b)]
    assert np.array_equal(y[..., keep], x[..., keep])
    # Rotations keep the length of a head, and a scale multiplies its rotated part.
    inv = 10.0 ** -np.arange(32)
    y, _ = oracle.norm_rotate(x, inv_freq=inv, positions=[[5, 700, -3]], interleaved=interleaved, scale=2.0)
    assert np.allclose((y * y).sum(-1), 4 * (x * x).sum(-1))
