"""Pins of the 8-bit checkpoint oracle: the exponent rule by brute force and by
its closed form at the borders, decoded values exact in bf16, half a step of
rounding, and agreement with torch's E4M3 cast."""

import math

import numpy as np
import torch

from oracle import act8
from oracle.numerics import bf16_bits_to_f32, f32_to_bf16_bits


def _bits(x):
    return f32_to_bf16_bits(np.asarray(x, dtype=np.float32))


def test_exponent_of_every_positive_bf16():
    """Every finite magnitude: a <= 448 2^e, and e - 1 would be too small."""
    b = np.arange(0, 0x7F80, dtype=np.uint16)
    a = bf16_bits_to_f32(b).astype(np.float64)
    e = act8.exponent(a)
    assert np.all(a <= np.ldexp(448.0, e))
    inner = e > act8.E_MIN
    assert np.all(a[inner] > np.ldexp(448.0, e[inner] - 1))
    assert e.min() == act8.E_MIN and e.max() == act8.E_MAX and e[0] == act8.E_MIN


def test_exponent_borders():
    assert act8.exponent(448.0) == 0 and act8.exponent(450.0) == 1
    assert act8.exponent(224.0) == -1 and act8.exponent(1.0) == -8 and act8.exponent(1.75) == -8
    assert act8.exponent(1.7578125) == -7


def test_decoded_values_are_exact_in_bf16():
    """Every finite code with every exponent byte a block can get, but for the
    magnitudes at 2^128, where bf16 ends."""
    codes = np.array([c for c in range(256) if c & 0x7F != 0x7F], dtype=np.uint8)
    for e in range(act8.E_MIN, act8.E_MAX + 1):
        v = act8.dequantize(np.resize(codes, (1, 256)), np.full((1, 4), e + 127, dtype=np.uint8)).reshape(-1)
        v = v[np.abs(v) < 2.0 ** 128]
        back = bf16_bits_to_f32(f32_to_bf16_bits(v.astype(np.float32))).astype(np.float64)
        assert np.array_equal(back, v)


def test_rounding_is_at_most_half_a_step():
    rng = np.random.default_rng(0)
    x = _bits(rng.standard_normal((64, 256)) * np.exp(rng.uniform(-8, 8, (64, 1))))
    codes, exps = act8.quantize(x)
    v, ref = act8.dequantize(codes, exps), bf16_bits_to_f32(x).astype(np.float64)
    smallest = np.repeat(np.ldexp(1.0, exps.astype(int) - 127 - 10), 64, axis=1)  # half the subnormal step
    assert np.all(np.abs(v - ref) <= np.maximum(2.0 ** -4 * np.abs(ref), smallest))
    again, e2 = act8.quantize(_bits(v))
    assert np.array_equal(act8.dequantize(again, e2), v)  # a checkpoint of its own values is itself


def test_codes_equal_torch_cast():
    rng = np.random.default_rng(1)
    x = _bits(rng.standard_normal((32, 192)) * 3.0)
    codes, exps = act8.quantize(x)
    scaled = torch.from_numpy(np.ldexp(bf16_bits_to_f32(x).reshape(32, 3, 64), -(exps.astype(int) - 127)[..., None]))
    want = scaled.to(torch.float8_e4m3fn).view(torch.uint8).numpy().reshape(32, 192)
    assert np.array_equal(codes, want)


def test_extremes():
    z = np.zeros((1, 64), dtype=np.float32)
    codes, exps = act8.quantize(_bits(z))
    assert not codes.any() and exps[0, 0] == act8.E_MIN + 127
    z[0, 0], z[0, 1] = 2.0 ** 127 * 1.5, -math.ldexp(1, -126)
    codes, exps = act8.quantize(_bits(z))
    assert exps[0, 0] == act8.E_MAX + 127 - 1 and act8.dequantize(codes, exps)[0, 0] == 2.0 ** 127 * 1.5
    assert codes[0, 1] == 0x80  # rounds to zero, sign kept
    assert act8.quantize(np.zeros((0, 64), dtype=np.uint16))[0].shape == (0, 64)
