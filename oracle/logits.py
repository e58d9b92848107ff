"""Plain CPU oracle of the operators on logits (float64 numpy).

TEST INFRASTRUCTURE ONLY: only the tests use it; it shares no code with the
CUDA library.

A row of logits x gives p = softmax(scale x).  A logit of -inf is a masked
token.  Rows that are left out (a negative token; no teacher entry) give 0; a
row of nothing but -inf has log probability -inf, entropy 0, gradient 0.
"""
from __future__ import annotations

import numpy as np


def row_log_softmax(x, scale):
    """ln p per row; -inf everywhere in a row of nothing but -inf."""
    m = np.max(x, axis=1, keepdims=True)
    empty = np.isneginf(m)
    z = (x - np.where(empty, 0.0, m)) * scale
    total = np.sum(np.exp(z), axis=1, keepdims=True)
    return z - np.log(np.where(empty, 1.0, total))


def xlogx(lp):
    """p ln p with 0 ln 0 = 0."""
    p = np.exp(lp)
    return np.where(p > 0, p * np.where(np.isneginf(lp), 0.0, lp), 0.0)


def token_logprobs(x, tokens, topk, scale):
    """(logp, entropy, top_tokens, top_logp); tokens may be None (logp is None then)."""
    T, V = x.shape
    lp = row_log_softmax(x, scale)
    H = -xlogx(lp).sum(axis=1)
    live = np.ones(T, bool) if tokens is None else tokens >= 0
    logp = None if tokens is None else np.where(live, lp[np.arange(T), np.maximum(tokens, 0)], 0.0)
    top = np.full((T, topk), -1, np.int64)
    topl = np.full((T, topk), -np.inf)
    for t in range(T):
        if live[t] and topk:
            order = np.argsort(-x[t], kind="stable")[:topk]
            order = order[x[t][order] > -np.inf]
            top[t, :len(order)] = order
            topl[t, :len(order)] = lp[t][order]
    return logp, np.where(live, H, 0.0), top, topl


def token_logprobs_grad(x, tokens, dlogp, dentropy, scale):
    """The gradient of sum dlogp logp + dentropy entropy with respect to x, and the magnitude of its terms."""
    T, V = x.shape
    lp = row_log_softmax(x, scale)
    p = np.exp(lp)
    d, mag = np.zeros((T, V)), np.zeros((T, V))
    if dlogp is not None:
        d -= dlogp[:, None] * p
        mag += np.abs(dlogp)[:, None] * p
        hot = np.zeros((T, V))
        hot[np.arange(T), np.maximum(tokens, 0)] = 1.0
        d += dlogp[:, None] * hot
        mag += np.abs(dlogp)[:, None] * hot
    if dentropy is not None:
        H = -xlogx(lp).sum(axis=1, keepdims=True)
        d -= dentropy[:, None] * (xlogx(lp) + p * H)
        mag += np.abs(dentropy)[:, None] * (np.abs(xlogx(lp)) + p * H)
    dead = np.all(np.isneginf(x), axis=1)
    if tokens is not None:
        dead |= tokens < 0
    d[dead], mag[dead] = 0.0, 0.0
    return d * scale, mag * scale


def _teacher(tokens, values, value_scale, tail):
    """q and ln q of one row's entries, q_r, or None when no entry counts."""
    u = np.where(tokens >= 0, values * value_scale, -np.inf)
    if not np.any(tokens >= 0) or (not tail and np.all(np.isneginf(u))):
        return None
    if tail:
        lq, rest = u, max(0.0, 1.0 - np.exp(u).sum())
        if rest < np.sum(tokens >= 0) * 2.0 ** -23:
            rest = 0.0
    else:
        lq = u - u.max()
        lq, rest = lq - np.log(np.exp(lq).sum()), 0.0
    return np.exp(lq), lq, rest


def distill(x, tokens, values, dloss=None, value_scale=1.0, tail=False, scale=1.0):
    """(loss, dlogits, magnitude of the gradient's terms) against the teacher's entries."""
    T, V = x.shape
    lp = row_log_softmax(x, scale)
    p = np.exp(lp)
    loss, d, mag = np.zeros(T), np.zeros((T, V)), np.zeros((T, V))
    for t in range(T):
        teacher = _teacher(tokens[t], values[t], value_scale, tail)
        if teacher is None:
            continue
        q, lq, rest = teacher
        use = q > 0
        loss[t] = np.sum(q[use] * (lq[use] - lp[t][tokens[t][use]]))
        inside = np.zeros(V, bool)
        inside[tokens[t][tokens[t] >= 0]] = True
        qd = np.zeros(V)
        np.add.at(qd, tokens[t][use], q[use])
        g = (1.0 if dloss is None else dloss[t]) * scale
        # every ln p of the loss takes p along with it, once for each part of the mass that the loss counts
        mass = q.sum() + (rest if tail and not inside.all() else 0.0)
        row, m = p[t] * mass - qd, p[t] * mass + qd
        if tail and not inside.all():
            pr = p[t][~inside].sum()
            if rest > 0:
                with np.errstate(divide="ignore"):
                    loss[t] += rest * (np.log(rest) - np.log(pr))
            if pr > 0:
                row = np.where(inside, row, p[t] / pr * (pr * mass - rest))
                m = np.where(inside, m, p[t] / pr * (pr * mass + rest))
            else:
                row, m = np.where(inside, row, 0.0), np.where(inside, m, 0.0)
        if np.all(np.isneginf(x[t])):
            row, m = np.zeros(V), np.zeros(V)
        d[t], mag[t] = row * g, m * abs(g)
    return loss, d, mag
