"""Oracle for the operators over rows of logits.

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py).

Plain float64 definitions, one row at a time, of what include/ws_logits.h
documents: log probabilities, entropy, the best alternatives, distillation
losses against a teacher's listed entries, and the gradients of all of them.
Rows without a distribution follow the header's rules: a row of -inf only has
log probabilities -inf, entropy 0 and gradient 0; a NaN or +inf makes the
row's results NaN; an index of -1 is no token, and any other index outside the
row makes what depends on it NaN.  A teacher's q_t of at most ROUNDING counts as
0 where p_t is 0 in FP32.
"""
from __future__ import annotations

import numpy as np

RENORM = 0
TAIL = 1
ROUNDING = 2.0 ** -16
LOG_NONE = -150 * np.log(2.0)      # log p_t below which p_t is 0 in FP32


def log_softmax(z, tau):
    """Row log probabilities in float64 (NaN for a row with NaN or +inf)."""
    z = np.asarray(z, dtype=np.float64)
    if np.isnan(z).any() or np.isposinf(z).any():
        return np.full(z.shape, np.nan)
    m = z.max()
    if np.isneginf(m):
        return np.full(z.shape, -np.inf)
    d = (z - m) / tau
    return d - np.log(np.exp(d).sum())


def entropy(logp):
    p = np.exp(logp)
    return float(-(p[p > 0] * logp[p > 0]).sum()) if not np.isnan(logp).any() else np.nan


def best(z, k):
    """Indices of the k best logits: value descending, index ascending, NaN as
    -inf, -0 equal to +0 (a full stable sort)."""
    v = np.where(np.isnan(z), -np.inf, np.asarray(z, dtype=np.float64))
    return np.argsort(-v, kind="stable")[:k]


def stats(z, tau):
    """(max, log sum exp((z - max) / tau)) of a row."""
    z = np.asarray(z, dtype=np.float64)
    m = z.max()
    if np.isneginf(m):
        return -np.inf, -np.inf
    if not np.isfinite(m):
        return m, np.nan
    return m, np.log(np.exp((z - m) / tau).sum())


def token_logprob(logp, t):
    if t == -1:
        return 0.0
    return logp[t] if 0 <= t < len(logp) else np.nan


def logprobs_grad(z, tau, target=-1, g_target=0.0, g_entropy=0.0, ids=(), g_ids=()):
    """d(g_target logprob + g_entropy entropy + sum g_ids top) / dz of a row."""
    logp = log_softmax(z, tau)
    n = len(logp)
    named = [(target, g_target)] if target != -1 else []
    named += [(i, g) for i, g in zip(ids, g_ids) if i != -1]
    if np.isnan(logp).any() or any(not 0 <= i < n for i, _ in named):
        return np.full(n, np.nan)
    if np.isneginf(logp).all():
        return np.zeros(n)
    p = np.exp(logp)
    dx = np.zeros(n)
    for i, g in named:
        dx[i] += g
        dx -= g * p
    bend = np.where(p > 0, p * (np.where(p > 0, logp, 0.0) + entropy(logp)), 0.0)
    return (dx - g_entropy * bend) / tau


def teacher_weights(scores, ids, vocab, mode):
    """(q per entry, log q per entry, q_t) of one row's teacher entries."""
    scores = np.asarray(scores, dtype=np.float64)
    there = np.asarray(ids) != -1
    logq = np.where(there, scores, -np.inf)
    rest = 0.0
    if mode == RENORM:
        if there.any() and not np.isneginf(logq).all():
            high = logq.max()
            logq = logq - (high + np.log(np.exp(logq - high).sum()))
    elif len(set(np.asarray(ids)[there].tolist())) < vocab:
        rest = max(0.0, 1.0 - np.exp(logq).sum())
    return np.exp(logq), logq, rest


def distill(z, tau, scores, ids, mode, g=1.0):
    """(loss, d(g loss)/dz, log p_t) of one row."""
    logp = log_softmax(z, tau)
    n = len(logp)
    ids = np.asarray(ids)
    there = ids != -1
    bad = ((ids[there] < 0) | (ids[there] >= n)).any()
    if bad or np.isnan(logp).any():
        return np.nan, np.full(n, np.nan), np.nan
    q, logq, rest = teacher_weights(scores, ids, n, mode)
    loss = sum(q[k] * (logq[k] - logp[ids[k]]) for k in range(len(ids)) if q[k] > 0)
    p = np.exp(logp)
    outside = np.ones(n, dtype=bool)
    outside[ids[there]] = False
    tail = np.nan
    spread = np.zeros(n)
    np.add.at(spread, ids[there], q[there])
    if mode == TAIL:
        left = logp[outside]
        tail = -np.inf
        if left.size and not np.isneginf(left).all():
            tail = left.max() + np.log(np.exp(left - left.max()).sum())
        if rest <= ROUNDING and tail < LOG_NONE:
            rest = 0.0
        if rest > 0:
            loss += rest * (np.log(rest) - tail)
            if not np.isneginf(tail):
                spread += rest * np.exp(np.where(outside, logp - tail, -np.inf))
    grad = g / tau * ((q.sum() + rest) * p - spread)
    if np.isneginf(logp).all():
        grad = np.zeros(n)
    return float(loss), grad, tail
