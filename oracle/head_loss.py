"""Softmax cross entropy of the head's logits and its gradient (test
infrastructure only), in fp64 on the exact bf16 inputs, with the logits written
out.

    l = H W^T;  lse = log sum exp l;  loss = lse - l[label] (0 if ignored)
    mean = sum loss / count (0 if count = 0)
    dH_t = g_t (softmax(l_t) - onehot(label_t)) W

Parity status: pinned (textbook closed forms, shift invariance and central
differences in tests/test_oracle_head_loss.py).
"""

import numpy as np

from .numerics import bf16_bits_to_f32


def _f64(bits):
    return bf16_bits_to_f32(bits).astype(np.float64)


def counted(labels, vocab, ignore_index=-100):
    labels = np.asarray(labels)
    return (labels != ignore_index) & (labels >= 0) & (labels < vocab)


def fwd(h_bits, w_bits, labels, ignore_index=-100):
    """Returns (loss [T], lse [T], mean, count)."""
    z = _f64(h_bits) @ _f64(w_bits).T
    top = z.max(axis=1, keepdims=True)
    lse = np.log(np.exp(z - top).sum(axis=1)) + top[:, 0]
    c = counted(labels, w_bits.shape[0], ignore_index)
    loss = np.zeros(z.shape[0])
    i = np.nonzero(c)[0]
    loss[i] = lse[i] - z[i, np.asarray(labels)[i]]
    n = int(c.sum())
    return loss, lse, (loss.sum() / n if n else 0.0), n


def probabilities(h_bits, w_bits, labels, ignore_index=-100):
    """softmax(l) - onehot(label), zero rows for ignored tokens: [T, vocab]."""
    z = _f64(h_bits) @ _f64(w_bits).T
    z = z - z.max(axis=1, keepdims=True)
    p = np.exp(z)
    p /= p.sum(axis=1, keepdims=True)
    c = counted(labels, w_bits.shape[0], ignore_index)
    i = np.nonzero(c)[0]
    y = np.asarray(labels)[i]
    others = p[i].copy()
    others[np.arange(i.size), y] = 0.0
    p[i, y] = -others.sum(axis=1)  # p - 1 without the cancellation
    p[~c] = 0.0
    return p


def bwd(h_bits, w_bits, labels, g, ignore_index=-100):
    """dH [T, dim] for per-token loss gradients g [T]."""
    p = probabilities(h_bits, w_bits, labels, ignore_index)
    g = np.where(counted(labels, w_bits.shape[0], ignore_index), np.asarray(g, dtype=np.float64), 0.0)
    return (p * g[:, None]) @ _f64(w_bits)
