"""Plain forms of the mixture-of-experts operators in float64, and MXFP4 matrices for their tests (NumPy)."""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6])


def matrix(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """What nibble codes [..., K/2] (element 2j low) and E8M0 codes [..., K/32] stand for."""
    q = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    return E2M1[q] * np.repeat(2.0 ** (scales.astype(np.float64) - 127), 32, axis=-1)


def rotate(x: np.ndarray, b: int) -> np.ndarray:
    h = np.ones((1, 1))
    while len(h) < b:
        h = np.block([[h, h], [h, -h]])
    return (x.reshape(-1, b) @ h / np.sqrt(b)).reshape(x.shape)


def route(x: np.ndarray, w: np.ndarray):
    """(logits, softmax) in float64."""
    z = x.astype(np.float64) @ w.astype(np.float64).T
    p = np.exp(z - z.max(1, keepdims=True))
    return z, p / p.sum(1, keepdims=True)


def experts(x, ids, weights, w13, w2, block):
    """y and, per element, the sum of magnitudes it is made of: [T, D] float64. w13 [E, 2I, D], w2 [E, D, I]."""
    x = rotate(x.astype(np.float64), block)
    T, D = x.shape
    E, I = w2.shape[0], w2.shape[2]
    y, size = np.zeros((T, D)), np.zeros((T, D))
    for t in range(T):
        for e, p in zip(ids[t], weights[t].astype(np.float64)):
            if not 0 <= e < E:
                continue
            u = w13[e] @ x[t]
            s = np.abs(w13[e]) @ np.abs(x[t])  # magnitudes behind gate and up
            a, c = u[:I], u[I:]
            sig = 1 / (1 + np.exp(-a))
            h = a * sig * c
            # d(silu(a) c) <= 1.1 |c| da + |silu(a)| dc
            sh = 1.1 * np.abs(c) * s[:I] + np.abs(a * sig) * s[I:]
            y[t] += p * (w2[e] @ rotate(h, block))
            size[t] += abs(p) * (np.abs(w2[e]) @ rotate_abs(sh + np.abs(h), block))
    return y, size


def rotate_abs(v: np.ndarray, b: int) -> np.ndarray:
    """Bound of a rotated vector by the magnitudes of its block."""
    return np.repeat(v.reshape(-1, b).sum(1, keepdims=True) / np.sqrt(b), b, 1).reshape(v.shape)
