"""Oracle for the operators over rows of hidden states.

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py).

Plain float64 definitions of what include/ws_states.h documents: embedding
lookup with scaling and its gradient, layer norm and its gradients.
"""
from __future__ import annotations

import numpy as np


def embed(table, ids, scale):
    """scale * table[id] a row; 0 for -1, NaN for any other index outside."""
    table = np.asarray(table, dtype=np.float64)
    out = np.zeros((len(ids), table.shape[1]))
    for r, i in enumerate(ids):
        if 0 <= i < len(table):
            out[r] = scale * table[i]
        elif i != -1:
            out[r] = np.nan
    return out


def embed_grad(grad, ids, vocab, scale, held=None):
    """The sum of every token's rows, scaled; added to `held` if given."""
    grad = np.asarray(grad, dtype=np.float64)
    out = np.zeros((vocab, grad.shape[1]))
    for r, i in enumerate(ids):
        if 0 <= i < vocab:
            out[i] += grad[r]
    out *= scale
    return out if held is None else out + np.asarray(held, dtype=np.float64)


def norm_stats(x, eps):
    """(mean, 1 / sqrt(variance + eps)) of every row."""
    x = np.asarray(x, dtype=np.float64)
    mean = x.mean(1)
    var = ((x - mean[:, None]) ** 2).mean(1)
    with np.errstate(divide="ignore"):
        return mean, 1.0 / np.sqrt(var + eps)


def layernorm(x, weight, bias, eps):
    x = np.asarray(x, dtype=np.float64)
    mean, inverse = norm_stats(x, eps)
    y = (x - mean[:, None]) * inverse[:, None]
    if weight is not None:
        y = y * np.asarray(weight, dtype=np.float64)
    if bias is not None:
        y = y + np.asarray(bias, dtype=np.float64)
    return y


def layernorm_grad(x, mean, inverse, weight, grad):
    """(grad_x, grad_weight, grad_bias) with the statistics as given."""
    x, grad = np.asarray(x, dtype=np.float64), np.asarray(grad, dtype=np.float64)
    u = (x - mean[:, None]) * inverse[:, None]
    d = grad if weight is None else grad * np.asarray(weight, dtype=np.float64)
    level = d.mean(1, keepdims=True)
    along = (d * u).mean(1, keepdims=True)
    return inverse[:, None] * (d - level - u * along), (grad * u).sum(0), grad.sum(0)
