"""Norm and clip over a list of tensors, fp64 CPU reference.

``norm = sqrt(sum_t sum_i x_ti^2)`` or ``max |x_ti|``; a NaN anywhere gives
NaN, else an infinity gives infinity.  ``c = max_norm / norm`` when the norm is
finite and greater than ``max_norm``, else 1 (the clip rule of ``budget``).
"""
import math

import numpy as np

L2, MAX = 0, 1


def norm(tensors, kind=L2):
    parts = [np.asarray(t, dtype=np.float64).ravel() for t in tensors]
    x = np.concatenate(parts) if parts else np.zeros(0)
    if x.size == 0:
        return 0.0
    if np.any(np.isnan(x)):
        return float("nan")
    if kind == MAX:
        return float(np.max(np.abs(x)))
    if np.any(np.isinf(x)):
        return float("inf")
    return math.sqrt(math.fsum(x * x)) if x.size <= 1 << 16 else float(np.sqrt(np.sum(x * x)))


def clip(tensors, max_norm, kind=L2):
    """(norm, c, [c * t in fp64 ...])"""
    n = norm(tensors, kind)
    c = max_norm / n if np.isfinite(n) and n > max_norm else 1.0
    return n, c, [np.asarray(t, dtype=np.float64) * c for t in tensors]
