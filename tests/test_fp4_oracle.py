"""Pins of the 4-bit pool's oracle and of the rotation's (CPU)."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import fp4_oracle as f4


def test_scale_bytes_are_the_upper_bits_of_an_f16():
    bits = (np.arange(256, dtype=np.uint16) << 7).view(np.float16).astype(np.float64)
    t = f4.scale_table()
    same = (t == bits) | (np.isnan(t) & np.isnan(bits))
    assert same.all()
    assert t[248 - 1] == 61440.0 and (6 * 10240.0) in t


def test_every_value_is_an_f16_value():
    t = f4.scale_table()
    for s in t[:248][t[:248] <= f4.MAX_SCALE]:
        v = f4.E2M1 * s
        assert np.array_equal(v.astype(np.float16).astype(np.float64), v)


@pytest.mark.parametrize("spread", [0.0, 1.0, 4.0])
def test_quantisation_is_the_nearest_value(spread):
    rng = np.random.default_rng(int(spread) + 3)
    x = (rng.standard_normal((300, 64)) * np.exp(spread * rng.standard_normal((300, 1)))).astype(np.float32)
    x[0] = 0
    codes, scales = f4.quantize(x)
    v = f4.dequantize(codes, scales)
    s = np.repeat(f4.scale_table()[scales], 16, axis=-1)
    # no other code of the block's scale is nearer
    best = np.abs(np.abs(x)[..., None] - s[..., None] * f4.E2M1).min(-1)
    assert np.allclose(np.abs(x - v), best, rtol=0, atol=1e-6 * np.abs(x).max())
    # the scale is the nearest to amax / 6 of all that are at most 10240
    raw = np.minimum(np.abs(x).reshape(300, 4, 16).max(-1) / np.float32(6), np.float32(10240)).astype(np.float64)
    t = f4.scale_table()[:248]
    near = np.abs(raw[..., None] - t[t <= f4.MAX_SCALE]).min(-1)
    assert np.array_equal(np.abs(raw - t[scales]), near)
    assert (scales[0] == 0).all() and (codes[0] == 0).all()


def test_ties_saturation_and_non_finite_blocks():
    x = np.zeros((6, 16), np.float32)
    x[0] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5, -6]   # scale 1
    codes, scales = f4.quantize(x[:1])
    assert scales[0, 0] == 15 << 3
    got = f4.dequantize(codes, scales)[0]
    assert got.tolist() == [6, 0, 1, 1, 2, 2, 4, 4, 0, -1, -1, -2, -2, -4, -4, -6]
    x[1] = 1e30
    x[2, 3] = np.inf
    x[3, 5] = np.nan
    x[4] = 2.0 ** -20          # amax / 6 rounds to scale 0
    x[5] = 6 * 2.0 ** -17      # the smallest scale
    codes, scales = f4.quantize(x)
    v = f4.dequantize(codes, scales)
    assert (v[1] == 61440).all()
    assert scales[2, 0] == 255 and scales[3, 0] == 255 and np.isnan(v[2]).all() and np.isnan(v[3]).all()
    assert scales[4, 0] == 0 and (codes[4] == 0).all()
    assert scales[5, 0] == 1 and (v[5] == 6 * 2.0 ** -17).all()


def test_nibble_order():
    x = np.zeros((1, 16), np.float32)
    x[0, 0], x[0, 1], x[0, 15] = 6.0, 1.0, -6.0
    codes, _ = f4.quantize(x)
    assert codes[0, 0] == (7 | (2 << 4)) and codes[0, 7] == (15 << 4)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,rot,off", [(64, 64, 0), (128, 64, 0), (576, 64, 512), (128, 96, 16)])
def test_rotation_keeps_lengths_and_matches_64_bits(d, rot, off, inter):
    rng = np.random.default_rng(d + rot)
    x = rng.standard_normal((20, 3, d)).astype(np.float32)
    pos = rng.integers(0, 1000, 20)
    inv = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    a = np.arange(1000)[:, None] * inv
    table = np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)
    y, z = f4.rotate(x, table, pos, off, inter), f4.rotate64(x, table, pos, off, inter)
    assert np.abs(y - z).max() <= 4 * 2.0 ** -24 * 2 * np.abs(x).max()
    assert np.array_equal(y[..., :off], x[..., :off]) and np.array_equal(y[..., off + rot:], x[..., off + rot:])
    assert np.allclose((z ** 2).sum(-1), (x.astype(np.float64) ** 2).sum(-1), rtol=1e-5)
    zero = f4.rotate(x, table, np.zeros(20, np.int64), off, inter)
    assert np.array_equal(zero, x)
