"""Pins of the loss-head oracle: closed forms, shift invariance, ignored
tokens, and the gradient against central differences of the loss."""

import numpy as np

from oracle import head_loss as hl
from oracle.numerics import f32_to_bf16_bits


def _case(T=5, V=37, D=16, seed=0):
    rng = np.random.default_rng(seed)
    h = f32_to_bf16_bits(rng.standard_normal((T, D)).astype(np.float32))
    w = f32_to_bf16_bits((rng.standard_normal((V, D)) * 0.5).astype(np.float32))
    return h, w, rng.integers(0, V, T)


def test_uniform_logits():
    h, w, y = _case()
    loss, lse, mean, n = hl.fwd(np.zeros_like(h), w, y)
    assert n == 5 and np.allclose(loss, np.log(37.0)) and np.isclose(mean, np.log(37.0)) and np.allclose(lse, loss)
    p = hl.probabilities(np.zeros_like(h), w, y)
    assert np.allclose(p[0].sum(), 0.0) and np.isclose(p[0, y[0]], 1 / 37 - 1)


def test_two_classes_are_a_logistic():
    h = f32_to_bf16_bits(np.array([[2.0] + [0.0] * 7], dtype=np.float32))
    w = f32_to_bf16_bits(np.array([[1.5] + [0.0] * 7, [-0.5] + [0.0] * 7], dtype=np.float32))
    loss, _, _, _ = hl.fwd(h, w, [1])
    assert np.isclose(loss[0], np.log1p(np.exp(4.0)))


def test_ignored_and_out_of_range_tokens():
    h, w, y = _case()
    y = y.copy()
    y[1], y[3] = -100, 37
    loss, _, mean, n = hl.fwd(h, w, y)
    assert n == 3 and loss[1] == 0 and loss[3] == 0 and np.isclose(mean, loss.sum() / 3)
    d = hl.bwd(h, w, y, np.ones(5))
    assert not d[1].any() and not d[3].any() and d[0].any()
    assert hl.fwd(h, w, np.full(5, -100))[2:] == (0.0, 0)


def test_gradient_against_differences():
    h, w, y = _case(seed=3)
    g = np.linspace(-1, 2, 5)
    W = hl._f64(w)
    H = hl._f64(h)

    def total(H):
        z = H @ W.T
        lse = np.log(np.exp(z).sum(1))
        return float((g * (lse - z[np.arange(5), y])).sum())

    d = hl.bwd(h, w, y, g)
    for t, k in [(0, 0), (2, 7), (4, 15)]:
        e = np.zeros_like(H)
        e[t, k] = 1e-5
        num = (total(H + e) - total(H - e)) / 2e-5
        assert abs(num - d[t, k]) <= 1e-8 * max(1.0, abs(num)) * 10
