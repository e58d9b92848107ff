"""Plain CPU oracle of the joint between two blocks (float64 numpy).

TEST INFRASTRUCTURE ONLY: only the tests use it; it shares no code with the
CUDA library.

    p  = o / sqrt(mean(o^2) + eps) * w_post      (post_norm; otherwise p = o)
    h' = alpha h + beta act(g) p
    n  = h' / sqrt(mean(h'^2) + eps) * w_pre

Token t takes gate row t // gate_rows.  The backward is the chain rule written
out; the tests pin it against central differences.  Beside each gradient it
returns the sum of the magnitudes of the terms it is made of, which rounding
errors of a float computation are relative to.
"""
from __future__ import annotations

import numpy as np


def rms(x, eps):
    return np.sqrt(np.mean(x * x, axis=1, keepdims=True) + eps)


def gate_rows_of(gate, T, rows, sigmoid):
    """The gate of each token after its activation: T x d or T x 1 (ones without a gate)."""
    if gate is None:
        return np.ones((T, 1))
    g = gate.reshape(gate.shape[0], -1)[np.arange(T) // rows]
    return 1.0 / (1.0 + np.exp(-g)) if sigmoid else g


def forward(o, h, gate=None, w_post=None, w_pre=None, post_norm=True, sigmoid=False, rows=1, alpha=1.0, beta=1.0,
            eps=1e-6):
    """(h', n) and the magnitudes of their terms."""
    T, d = h.shape
    if o is None:
        after, mag = h, np.abs(h)
    else:
        p = o / rms(o, eps) * (1.0 if w_post is None else w_post) if post_norm else o
        a = gate_rows_of(gate, T, rows, sigmoid) * p
        after, mag = alpha * h + beta * a, np.abs(alpha * h) + np.abs(beta * a)
    r = rms(after, eps)
    w = 1.0 if w_pre is None else w_pre
    return after, after / r * w, mag, mag / r * np.abs(w) + np.abs(after / r * w)


def backward(o, after, gate, dh_out, dn, w_post=None, w_pre=None, post_norm=True, sigmoid=False, rows=1, alpha=1.0,
             beta=1.0, eps=1e-6):
    """{name: (gradient, magnitude of its terms)} for dh, do, dgate, dw_post, dw_pre."""
    ref = dh_out if dh_out is not None else dn
    T, d = ref.shape
    out = {}
    t, mt = (np.zeros((T, d)), np.zeros((T, d))) if dh_out is None else (dh_out, np.abs(dh_out))
    if dn is not None:
        r = rms(after, eps)
        nh = after / r
        u = dn * (1.0 if w_pre is None else w_pre)
        t = t + (u - nh * np.mean(u * nh, axis=1, keepdims=True)) / r
        mt = mt + (np.abs(u) + np.abs(nh) * np.mean(np.abs(u * nh), axis=1, keepdims=True)) / r
        out["dw_pre"] = (np.sum(dn * nh, axis=0), np.sum(np.abs(dn * nh), axis=0))
    if o is None:
        out["dh"] = (t, mt)
        return out
    out["dh"] = (alpha * t, abs(alpha) * mt)
    da, mda = beta * t, abs(beta) * mt
    if post_norm:
        ro = rms(o, eps)
        ph = o / ro
        w = 1.0 if w_post is None else w_post
    else:
        ro, ph, w = 1.0, o, 1.0
    g = gate_rows_of(gate, T, rows, sigmoid)
    dp, mdp = da * g, mda * np.abs(g)
    if gate is not None:
        deriv = g * (1.0 - g) if sigmoid else 1.0
        each, meach = da * ph * w * deriv, mda * np.abs(ph * w * deriv)
        if gate.ndim == 1:
            each, meach = each.sum(axis=1, keepdims=True), meach.sum(axis=1, keepdims=True)
        dg, mdg = np.zeros((gate.shape[0], each.shape[1])), np.zeros((gate.shape[0], each.shape[1]))
        np.add.at(dg, np.arange(T) // rows, each)
        np.add.at(mdg, np.arange(T) // rows, meach)
        out["dgate"] = (dg.reshape(gate.shape), mdg.reshape(gate.shape))
    if post_norm:
        out["dw_post"] = (np.sum(dp * ph, axis=0), np.sum(mdp * np.abs(ph), axis=0))
        v, mv = dp * w, mdp * np.abs(w)
        out["do"] = ((v - ph * np.mean(v * ph, axis=1, keepdims=True)) / ro,
                     (mv + np.abs(ph) * np.mean(mv * np.abs(ph), axis=1, keepdims=True)) / ro)
    else:
        out["do"] = (dp, mdp)
    return out
