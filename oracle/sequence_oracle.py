"""The sequence operators' definitions in float64 (NumPy, plain loops over time).

Independent of the library: event embedding, gated linear recurrence and token
log probabilities with their gradients, as include/symnmf.h states them.
"""
from __future__ import annotations

import numpy as np


def embed(table, ids, scale):
    """scale * table[ids]; negative ids give zeros, ids past the table NaN."""
    table = np.asarray(table, np.float64)
    ids = np.asarray(ids)
    out = np.zeros(ids.shape + (table.shape[1],))
    ok = (ids >= 0) & (ids < table.shape[0])
    out[ok] = scale * table[ids[ok]]
    out[ids >= table.shape[0]] = np.nan
    return out


def embed_grad(dout, ids, rows, scale):
    dout = np.asarray(dout, np.float64)
    out = np.zeros((rows, dout.shape[-1]))
    for i, v in enumerate(np.asarray(ids).reshape(-1)):
        if 0 <= v < rows:
            out[v] += scale * dout.reshape(-1, dout.shape[-1])[i]
    return out


def sigmoid(g):
    g = np.asarray(g, np.float64)
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-g))


def gated_scan(x, gate, h0=None, lengths=None):
    """(h with 0 at masked steps, the last state, the states before each step)."""
    x = np.asarray(x, np.float64)
    B, T, D = x.shape
    gate = np.broadcast_to(np.asarray(gate, np.float64), x.shape)
    n = np.full(B, T) if lengths is None else np.clip(lengths, 0, T)
    h = np.zeros((B, D)) if h0 is None else np.array(h0, np.float64)
    out = np.zeros_like(x)
    before = np.zeros((B, T + 1, D))
    for b in range(B):
        s = h[b].copy()
        for t in range(T):
            before[b, t] = s
            if t < n[b]:
                s = sigmoid(gate[b, t]) * s + sigmoid(-gate[b, t]) * x[b, t]
                out[b, t] = s
        before[b, T] = s
    return out, before[:, T].copy(), before


def gated_scan_grad(x, gate, dh, dlast=None, h0=None, lengths=None):
    """(dx, dgate, dh0), the gradients of sum(dh * h) + sum(dlast * last)."""
    x = np.asarray(x, np.float64)
    B, T, D = x.shape
    gate = np.broadcast_to(np.asarray(gate, np.float64), x.shape)
    n = np.full(B, T) if lengths is None else np.clip(lengths, 0, T)
    before = gated_scan(x, gate, h0, lengths)[2]
    dx, dg = np.zeros_like(x), np.zeros_like(x)
    m = np.zeros((B, D)) if dlast is None else np.array(dlast, np.float64)
    for b in range(B):
        for t in range(n[b] - 1, -1, -1):
            a, c = sigmoid(gate[b, t]), sigmoid(-gate[b, t])
            lam = np.asarray(dh[b, t], np.float64) + m[b]
            dx[b, t] = c * lam
            dg[b, t] = lam * (before[b, t] - x[b, t]) * a * c
            m[b] = a * lam
    return dx, dg, m


def log_softmax(logits, scale):
    """(ln p, lse, entropy); rows with nothing but -inf: -inf, -inf, 0."""
    z = np.asarray(logits, np.float64) * scale
    with np.errstate(invalid="ignore", divide="ignore"):
        m = z.max(axis=1, keepdims=True)
        m = np.where(np.isneginf(m), 0.0, m)
        e = np.exp(z - m)
        ls = np.log(e.sum(axis=1))
        lse = m[:, 0] + ls
        # not z - lse, which loses ls where m is of the order of 1e16 and more
        lp = np.where(np.isneginf(z), -np.inf, (z - m) - ls[:, None])
        p = np.exp(lp)
        h = -np.where(p > 0, p * lp, np.where(np.isnan(p), np.nan, 0.0)).sum(axis=1)
    return lp, lse, h


def token_logprobs(logits, tokens, top, scale):
    """(logp, entropy, lse, top_logp, top_ids)."""
    z = np.asarray(logits, np.float64)
    n, v = z.shape
    lp, lse, h = log_softmax(z, scale)
    tokens = np.asarray(tokens)
    logp = np.zeros(n)
    ok = (tokens >= 0) & (tokens < v)
    logp[ok] = lp[np.arange(n)[ok], tokens[ok]]
    logp[tokens >= v] = np.nan
    ids = np.full((n, top), -1, np.int64)
    tlp = np.full((n, top), -np.inf)
    order = np.argsort(-(z + 0.0), axis=1, kind="stable")[:, :top]
    got = np.take_along_axis(lp, order, 1)
    fine = ~np.isneginf(got)
    ids[:, :order.shape[1]] = np.where(fine, order, -1)
    tlp[:, :order.shape[1]] = got
    return logp, h, lse, tlp, ids


def token_logprobs_grad(logits, tokens, dlogp, dent, scale):
    lp, lse, h = log_softmax(logits, scale)
    n, v = lp.shape
    p = np.exp(lp)
    tokens = np.asarray(tokens)
    w = np.where(tokens >= 0, np.asarray(dlogp, np.float64), 0.0)
    q = np.zeros(n) if dent is None else np.asarray(dent, np.float64)
    flat = np.where(p > 0, p * (np.where(p > 0, lp, 0.0) + h[:, None]), 0.0)
    d = -w[:, None] * p - q[:, None] * flat
    ok = tokens >= 0
    d[np.arange(n)[ok], tokens[ok]] += w[ok]
    d[np.isneginf(lse)] = 0.0
    return scale * d
