"""The layer operators' definitions in float64 (NumPy, plain loops over time).

Independent of the library: linear attention with a decay for each head, rotary
positions and the AdamW step, as include/symnmf.h states them.
"""
from __future__ import annotations

import numpy as np


def _decays(decay):
    return np.exp(np.asarray(decay, np.float64))


def linear_attention(q, k, v, decay, state=None, lengths=None, scale=1.0):
    """(o with 0 at masked steps, the last state); q B x T x H x dk, k and v B x T x G x d."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    B, T, H, dk = q.shape
    G, dv = k.shape[2], v.shape[3]
    a = _decays(decay)
    n = np.full(B, T) if lengths is None else np.clip(lengths, 0, T)
    S = np.zeros((B, H, dk, dv)) if state is None else np.array(state, np.float64)
    o = np.zeros((B, T, H, dv))
    of = np.arange(H) // (H // G)
    for b in range(B):
        for t in range(n[b]):
            S[b] = a[:, None, None] * S[b] + k[b, t, of][:, :, None] * v[b, t, of][:, None, :]
            o[b, t] = scale * np.einsum("hi,hij->hj", q[b, t], S[b])
    return o, S


def linear_attention_grad(q, k, v, decay, do, dlast=None, state=None, lengths=None, scale=1.0):
    """(dq, dk, dv, dstate), the gradients of sum(do * o) + sum(dlast * last)."""
    q, k, v, do = (np.asarray(x, np.float64) for x in (q, k, v, do))
    B, T, H, dk_ = q.shape
    G, dv_ = k.shape[2], v.shape[3]
    a = _decays(decay)
    n = np.full(B, T) if lengths is None else np.clip(lengths, 0, T)
    of = np.arange(H) // (H // G)
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    R = np.zeros((B, H, dk_, dv_)) if dlast is None else np.array(dlast, np.float64)
    for b in range(B):
        S = np.zeros((H, dk_, dv_)) if state is None else np.array(state[b], np.float64)
        for t in range(n[b]):
            S = a[:, None, None] * S + k[b, t, of][:, :, None] * v[b, t, of][:, None, :]
            dq[b, t] = scale * np.einsum("hij,hj->hi", S, do[b, t])
        for t in range(n[b] - 1, -1, -1):
            R[b] += scale * q[b, t][:, :, None] * do[b, t][:, None, :]
            np.add.at(dk[b, t], of, np.einsum("hij,hj->hi", R[b], v[b, t, of]))
            np.add.at(dv[b, t], of, np.einsum("hij,hi->hj", R[b], k[b, t, of]))
            R[b] *= a[:, None, None]
    return dq, dk, dv, R


def rotary(x, positions, freqs, interleaved=False, amplitude=1.0, inverse=False):
    """x (..., heads, width) turned; angles in extended precision."""
    x = np.asarray(x, np.float64)
    angle = np.asarray(positions, np.longdouble)[..., None] * np.asarray(freqs, np.longdouble)
    angle = np.remainder(angle, 2 * np.arctan2(np.longdouble(0), np.longdouble(-1)))
    cos = (amplitude * np.cos(angle)).astype(np.float64)[..., None, :]
    sin = (amplitude * np.sin(angle)).astype(np.float64)[..., None, :]
    if inverse:
        sin = -sin
    half = len(freqs)
    out = x.copy()
    one, two = ((slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else
                (slice(0, half), slice(half, 2 * half)))
    out[..., one] = x[..., one] * cos - x[..., two] * sin
    out[..., two] = x[..., two] * cos + x[..., one] * sin
    return out


def adamw(p, g, m, v, step, lr, beta1, beta2, eps, weight_decay):
    """(p, m, v) after one step."""
    p, g, m, v = (np.asarray(x, np.float64) for x in (p, g, m, v))
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    with np.errstate(divide="ignore", invalid="ignore"):
        update = (m / (1 - beta1 ** step)) / (np.sqrt(v / (1 - beta2 ** step)) + eps)
    return p * (1 - lr * weight_decay) - lr * update, m, v
