"""The operators around the expert products, from their definitions (CPU oracle).

TEST INFRASTRUCTURE ONLY.  Nothing in the product path may import this file.

Residual addition + RMS norm, the router with its balance loss, the gradient
of the combine's weights and the gated activation, each with its gradient, in
float64.  Quantized outputs are not computed here: the quantization oracles
take these results.  ``tests/test_oracle_moe_ops.py`` holds every gradient
against differences of its forward.
"""
from __future__ import annotations

import numpy as np


def _f64(x):
    return np.asarray(x, np.float64)


# --- residual addition + RMS norm ---------------------------------------------

def add_rmsnorm(x, r, w, eps: float):
    """(a = x + r, rstd [T], y = a * rstd * w); r may be None."""
    a = _f64(x) if r is None else _f64(x) + _f64(r)
    rstd = 1.0 / np.sqrt(np.mean(a * a, axis=1) + eps)
    return a, rstd, a * rstd[:, None] * _f64(w)


def add_rmsnorm_grad(dy, a, rstd, w, dh=None):
    """(gradient of x and of r, gradient of w) from that of y and of a (dh)."""
    dy, a, rstd = _f64(dy), _f64(a), _f64(rstd)
    xh = a * rstd[:, None]
    g = dy * _f64(w)
    dx = rstd[:, None] * (g - xh * np.mean(g * xh, axis=1, keepdims=True))
    return dx if dh is None else dx + _f64(dh), np.sum(dy * xh, axis=0)


# --- router -------------------------------------------------------------------

def _live(logits, token_mask):
    x = np.array(logits, np.float64)
    if token_mask is not None:
        x[np.asarray(token_mask) == 0] = -np.inf
    return x


def scores(x, score: str):
    """(scores, probabilities of the balance loss) of logits x [T, E]."""
    if score == "softmax":
        m = np.max(x, axis=1, keepdims=True)
        e = np.exp(x - np.where(m == -np.inf, 0.0, m))
        z = e.sum(axis=1, keepdims=True)
        s = e / np.where(z == 0, 1.0, z)
        return s, s
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-x))
    z = s.sum(axis=1, keepdims=True)
    return s, s / np.where(z == 0, 1.0, z)


def choose(key, k: int):
    """The k largest keys of each row in descending order, ties to the lowest id."""
    return np.argsort(-key, axis=1, kind="stable")[:, :k]


def router(logits, k: int, score: str, renorm: bool, scale: float, bias=None, token_mask=None, idx=None):
    """dict of idx, w, counts [E], tokens, prob_sum, loss; a given idx is taken
    for the choice."""
    x = _live(logits, token_mask)
    T, E = x.shape
    s, p = scores(x, score)
    if idx is None:
        key = x if bias is None else np.where(x == -np.inf, -np.inf, s + _f64(bias))
        idx = choose(key, k)
    w = np.take_along_axis(s, idx, 1)
    if renorm:
        z = w.sum(axis=1, keepdims=True)
        w = w / np.where(z == 0, 1.0, z)
    live = np.take_along_axis(x, idx, 1) > -np.inf
    counts = np.bincount(idx[live], minlength=E)
    n = T if token_mask is None else int(np.count_nonzero(token_mask))
    psum = p.sum(axis=0)
    loss = E / (k * max(n, 1) ** 2) * float(np.dot(counts, psum))
    return dict(idx=idx, w=w * scale, counts=counts, tokens=n, prob_sum=psum, loss=loss, s=s, p=p)


def router_grad(logits, idx, counts, tokens: int, dw, dloss: float, score: str, renorm: bool, scale: float,
                token_mask=None):
    """Gradient of the logits from that of the weights (dw or None) and of the
    loss; the choice and the counts are constants."""
    x = _live(logits, token_mask)
    T, E = x.shape
    k = idx.shape[1]
    s, p = scores(x, score)
    c = dloss * E / (k * max(tokens, 1) ** 2) * _f64(counts)
    # gradient of p, then of s
    if score == "softmax":
        gs = np.broadcast_to(c, (T, E)).copy()
    else:
        z = s.sum(axis=1, keepdims=True)
        gs = (c - (p * c).sum(axis=1, keepdims=True)) / np.where(z == 0, 1.0, z)
    if dw is not None:
        d = _f64(dw) * scale
        sel = np.take_along_axis(s, idx, 1)
        if renorm:
            z = sel.sum(axis=1, keepdims=True)
            z = np.where(z == 0, 1.0, z)
            d = (d - (d * sel).sum(axis=1, keepdims=True) / z) / z
        for t in range(T):
            for j in range(k):
                gs[t, idx[t, j]] += d[t, j]
    out = s * (gs - (s * gs).sum(axis=1, keepdims=True)) if score == "softmax" else s * (1.0 - s) * gs
    return np.where(x == -np.inf, 0.0, out)


def weight_grad(dout, y, row_of):
    """dw[t, j] = <dout[t], y[row_of[t, j]]>; rows below 0 give 0."""
    dout, y = _f64(dout), _f64(y)
    out = np.zeros(row_of.shape)
    for t in range(row_of.shape[0]):
        for j in range(row_of.shape[1]):
            if row_of[t, j] >= 0:
                out[t, j] = np.dot(dout[t], y[row_of[t, j]])
    return out


# --- gated activation -----------------------------------------------------------

def _sig(g):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-g))


def swiglu(h):
    g, u = np.split(_f64(h), 2, axis=1)
    return g * _sig(g) * u


def swiglu_grad(dout, h):
    g, u = np.split(_f64(h), 2, axis=1)
    d, s = _f64(dout), _sig(g)
    return np.concatenate([d * u * s * (1.0 + g * (1.0 - s)), d * g * s], axis=1)


# --- the expert layer of a few tokens ---------------------------------------------

def moe_decode(x, idx, w, w1, w2, gamma: float = 0.0, act_rel: float = 0.0):
    """(out [T, H], bound): sum_j w[t, j] W2[e] swiglu(W1[e] x[t]) over the choices
    with 0 <= e < E and w != 0; w1 [E, 2F, H], w2 [E, H, F] values.  ``bound``:
    how far out may be off when every sum of products is known to gamma times
    the sum of their magnitudes and the activation to act_rel of itself."""
    x, w = _f64(x), _f64(w)
    T, H = x.shape
    E, _, F = w2.shape
    out, bound = np.zeros((T, H)), np.zeros((T, H))
    for e in range(E):
        t, j = np.nonzero((idx == e) & (w != 0))
        if not len(t):
            continue
        gu = x[t] @ w1[e].T
        d = gamma * (np.abs(x[t]) @ np.abs(w1[e]).T)
        g, u = gu[:, :F], gu[:, F:]
        with np.errstate(over="ignore", invalid="ignore"):
            s = g * _sig(g)
        a = s * u
        # |d silu| <= 1.1
        da = 1.1 * d[:, :F] * (np.abs(u) + d[:, F:]) + np.abs(s) * d[:, F:] + act_rel * np.abs(a)
        y, dy = a @ w2[e].T, (da + gamma * np.abs(a)) @ np.abs(w2[e]).T
        np.add.at(out, t, w[t, j][:, None] * y)
        np.add.at(bound, t, np.abs(w[t, j])[:, None] * (dy + gamma * np.abs(y)))
    return out, bound
