"""Orthogonalised updates, fp64 CPU reference.

``X = U / (|U|_F + eps)``, then ``steps`` times ``X <- a X + (b A + c A A) X`` with ``A = X
X^T`` on the smaller side; and the update of weights with momentum that uses it.

``noise``: a relative error of that size with random signs on every matrix that
enters a product and on every sum, which shows how far a rounding of the operands
moves the result.
"""
import numpy as np

A, B, C = 3.4445, -4.7750, 2.0315
SHAPE, RMS = 0, 1


def orthogonalize(u, steps=5, eps=1e-7, noise=0.0, seed=0):
    g = np.random.default_rng(seed)

    def off(x):
        return x * (1.0 + noise * g.choice([-1.0, 1.0], x.shape)) if noise else x

    u = np.asarray(u, np.float64)
    x = off(u / (np.linalg.norm(u) + eps))
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.T
    for _ in range(steps):
        s = off(x @ x.T)
        x = off(A * x + off(B * s + C * (s @ s)) @ x)
    return x.T if tall else x


def scalar(s, steps=5):
    """What becomes of a singular value."""
    for _ in range(steps):
        s = A * s + B * s ** 3 + C * s ** 5
    return s


def rate(lr, shape, scale=SHAPE):
    r, c = shape
    return lr * (max(1.0, r / c) ** 0.5 if scale == SHAPE else 0.2 * max(r, c) ** 0.5)


def muon(w, m, g, lr, mu=0.95, nesterov=True, weight_decay=0.0, scale=SHAPE, steps=5, eps=1e-7):
    """(weights, momentum) after one step"""
    w, m, g = (np.asarray(t, np.float64) for t in (w, m, g))
    m = mu * m + g
    u = g + mu * m if nesterov else m
    if not np.all(np.isfinite(u)):
        return w, None
    return (1.0 - lr * weight_decay) * w - rate(lr, w.shape, scale) * orthogonalize(u, steps, eps), m
