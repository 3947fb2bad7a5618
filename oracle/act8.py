"""8-bit activation checkpoints (test infrastructure only).

Reading of this library (the pages name memory as what the method saves and
fix no activation format): per row, blocks of 64 elements; e is the smallest
integer with max|x| <= 448 * 2**e, clamped to [-118, 120] (an all-zero block:
-118); the exponent byte is e + 127; the code is E4M3 (round to nearest even,
saturating) of x * 2**-e; a code stands for e4m3(code) * 2**e.

Written from those definitions with exact fp64 arithmetic: every bf16 value
times a power of two is exact, and the search for e compares exact products.

Parity status: pinned (brute force over the exponent, a closed-form table of
block maxima, and exactness of the decoded values in bf16, in
tests/test_oracle_act8.py).
"""

import numpy as np

from .numerics import bf16_bits_to_f32, e4m3_decode, e4m3_encode

BLOCK = 64
E_MIN, E_MAX = -118, 120


def exponent(amax):
    """Smallest e in [E_MIN, E_MAX] with amax <= 448 * 2**e (E_MAX if none)."""
    amax = np.asarray(amax, dtype=np.float64)
    e = np.full(amax.shape, E_MAX, dtype=np.int64)
    for cand in range(E_MAX, E_MIN - 1, -1):
        e = np.where(amax <= np.ldexp(448.0, cand), cand, e)
    return e


def quantize(x_bits):
    """bf16 bit patterns [M, K] (finite) -> (codes uint8 [M, K], exps uint8 [M, K/64])."""
    x = bf16_bits_to_f32(x_bits).astype(np.float64)
    M, K = x.shape
    b = x.reshape(M, K // BLOCK, BLOCK)
    e = exponent(np.abs(b).max(axis=-1)) if M else np.zeros((0, K // BLOCK), dtype=np.int64)
    scaled = np.ldexp(b, -e[..., None])
    # an fp32 holds every scaled value but those far below E4M3's smallest step,
    # which round to zero either way
    f32 = scaled.astype(np.float32)
    codes = e4m3_encode(f32) | np.where(np.signbit(f32), 0x80, 0).astype(np.uint8)  # the sign of a zero stays
    return codes.reshape(M, K).astype(np.uint8), (e + 127).astype(np.uint8)


def dequantize(codes, exps):
    """The fp64 values the codes stand for."""
    M, K = codes.shape
    v = e4m3_decode(codes).astype(np.float64).reshape(M, K // BLOCK, BLOCK)
    return np.ldexp(v, exps.astype(np.int64)[..., None] - 127).reshape(M, K)
