"""Softmax cross entropy of the actions taken under a linear policy head, with
its gradients, fp64 CPU reference.

``z = H W^T + b``, ``lse = log sum exp z`` over the actions, ``nll = lse - z[taken]``,
``loss = scale sum w nll``; rows whose action is outside of the actions, or whose
weight is 0, add nothing.  ``exp(-inf) = 0``: an action with a bias of minus
infinity is never taken.
"""
import numpy as np


def logits(hidden, weight, bias=None):
    z = np.asarray(hidden, np.float64) @ np.asarray(weight, np.float64).T
    return z if bias is None else z + np.asarray(bias, np.float64)[None, :]


def lse_of(z):
    top = z.max(axis=1)
    ref = np.where(np.isfinite(top), top, 0.0)
    with np.errstate(divide="ignore", invalid="ignore"):
        return ref + np.log(np.exp(z - ref[:, None]).sum(axis=1))


def on_rows(taken, actions, row_weights=None):
    taken = np.asarray(taken)
    there = (taken >= 0) & (taken < actions)
    return there, there if row_weights is None else there & (np.asarray(row_weights) != 0)


def loss(hidden, weight, taken, bias=None, row_weights=None, scale=1.0):
    """(loss, nll, lse)"""
    z = logits(hidden, weight, bias)
    lse = lse_of(z)
    there, on = on_rows(taken, z.shape[1], row_weights)
    at = np.where(there, taken, 0)
    za = z[np.arange(len(z)), at]
    with np.errstate(invalid="ignore"):
        nll = np.where(there, np.where(np.isneginf(za), np.inf, lse - za), 0.0)
    w = np.ones(len(z)) if row_weights is None else np.asarray(row_weights, np.float64)
    return scale * float(np.sum(w[on] * nll[on])), nll, lse


def logit_grads(hidden, weight, taken, bias=None, row_weights=None, scale=1.0):
    z = logits(hidden, weight, bias)
    lse = lse_of(z)
    _, on = on_rows(taken, z.shape[1], row_weights)
    p = np.exp(z - np.where(np.isneginf(lse), 0.0, lse)[:, None])
    w = np.ones(len(z)) if row_weights is None else np.asarray(row_weights, np.float64)
    p[np.arange(len(z))[on], np.asarray(taken)[on]] -= 1.0
    return np.where(on[:, None], scale * w[:, None] * p, 0.0)


def grads(hidden, weight, taken, bias=None, row_weights=None, scale=1.0):
    """(d_hidden, d_weight, d_bias)"""
    g = logit_grads(hidden, weight, taken, bias, row_weights, scale)
    _, on = on_rows(taken, g.shape[1], row_weights)
    return g @ np.asarray(weight, np.float64), g[on].T @ np.asarray(hidden, np.float64)[on], g.sum(axis=0)
