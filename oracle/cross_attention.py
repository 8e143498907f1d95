"""Attention of queries to keys and values of another length, and the norms of
queries and keys, in float64 numpy.

Written from the formulas, one sequence and one head at a time, without the
library.  The attention functions also return how far a bf16 pipeline with 32-bit
sums may be off, element by element, counted in half steps of a bf16 rounding
(2^-8 of the value): where P and dz become operands of a product, and where a
result is stored.
"""
from __future__ import annotations

import math

import numpy as np

from .attention_opt import F32_SLACK, HALF_BF16, rotary


# ------------------------------------------------------------------ sequences
def sequence_rows(n, rows, offsets=None, lens=None):
    """(first row, rows, real rows) of every sequence."""
    if offsets is None:
        offsets = [rows // n * i for i in range(n + 1)]
    out = []
    for i in range(n):
        first = min(max(offsets[i], 0), rows)
        slot = min(max(offsets[i + 1], first), rows) - first
        real = slot if lens is None else min(max(lens[i], 0), slot)
        out.append((first, slot, real))
    return out


def _weights(q, k, scale):
    z = (q @ k.T) * scale
    m = z.max(axis=1, keepdims=True)
    e = np.exp(z - m)
    l = e.sum(axis=1, keepdims=True)
    return e / l, (m + np.log(l))[:, 0], np.abs(z).max(axis=1, keepdims=True) + 1.0


def _heads(x, rows, h, d):
    return x[rows, h * d: (h + 1) * d]


def forward(q, k, v, q_seq, k_seq, heads, kv_heads, d, scale):
    """q [rows, heads d], k, v [rows, kv_heads d] -> o, lse [heads, rows], the
    tolerances of both, and which query rows belong to a sequence (others are
    left as they are)."""
    rows = q.shape[0]
    o, tol = np.zeros_like(q), np.full_like(q, 1e-30)
    lse, ltol = np.full((heads, rows), -np.inf), np.zeros((heads, rows))
    owned = np.zeros(rows, dtype=bool)
    for (q0, slot, nq), (k0, _, nk) in zip(q_seq, k_seq):
        owned[q0: q0 + slot] = True
        if not nq or not nk:
            continue
        rq, rk = slice(q0, q0 + nq), slice(k0, k0 + nk)
        for h in range(heads):
            g = h // (heads // kv_heads)
            c = slice(h * d, (h + 1) * d)
            vh = _heads(v, rk, g, d)
            p, lse[h, rq], size = _weights(_heads(q, rq, h, d), _heads(k, rk, g, d), scale)
            o[rq, c] = p @ vh
            # an exponent is off by the 32-bit error of its score
            ltol[h, rq] = F32_SLACK / 8 * size[:, 0]
            tol[rq, c] += (HALF_BF16 + F32_SLACK * size) * (p @ np.abs(vh)) + \
                HALF_BF16 * np.abs(o[rq, c])
    return o, lse, tol, ltol, owned


def backward(q, k, v, dout, q_seq, k_seq, heads, kv_heads, d, scale):
    """(dq, dk, dv), their tolerances, and the part of those which 32-bit
    arithmetic alone may be off (as in attention_opt)."""
    out = [np.zeros_like(x) for x in (q, k, v)]
    tol = [np.full_like(x, 1e-30) for x in (q, k, v)]
    t32 = [np.zeros_like(x) for x in (q, k, v)]
    for (q0, _, nq), (k0, _, nk) in zip(q_seq, k_seq):
        if not nq or not nk:
            continue
        rq, rk = slice(q0, q0 + nq), slice(k0, k0 + nk)
        for h in range(heads):
            g = h // (heads // kv_heads)
            qh, kh, vh, do = (_heads(q, rq, h, d), _heads(k, rk, g, d), _heads(v, rk, g, d),
                              _heads(dout, rq, h, d))
            p, _, size = _weights(qh, kh, scale)
            dp = do @ vh.T
            delta = ((p @ vh) * do).sum(axis=1, keepdims=True)
            dz = p * (dp - delta)
            rel = F32_SLACK * size
            # delta is formed from the stored O: one rounding of P and one of O
            ddelta = ((2 * HALF_BF16 + rel) * (p @ np.abs(vh)) * np.abs(do)).sum(axis=1,
                                                                                 keepdims=True)
            e32 = p * rel * (np.abs(do) @ np.abs(vh).T + np.abs(delta))
            e = HALF_BF16 * np.abs(dz) + p * ddelta + e32
            for n, (rows, at, val, err, err32) in enumerate((
                    (rq, h, (dz @ kh) * scale, (e @ np.abs(kh)) * scale, (e32 @ np.abs(kh)) * scale),
                    (rk, g, (dz.T @ qh) * scale, (e.T @ np.abs(qh)) * scale,
                     (e32.T @ np.abs(qh)) * scale),
                    (rk, g, p.T @ do, ((HALF_BF16 + rel) * p).T @ np.abs(do),
                     (p * rel).T @ np.abs(do)))):
                c = slice(at * d, (at + 1) * d)
                out[n][rows, c] += val
                tol[n][rows, c] += err * (1 + HALF_BF16)
                t32[n][rows, c] += err32
    return out, [t + HALF_BF16 * np.abs(x) for t, x in zip(tol, out)], t32


# ------------------------------------------------------------------ norms
def _moments(x, eps, centred):
    m = x.mean(axis=-1, keepdims=True) if centred else np.zeros(x.shape[:-1] + (1,))
    r = 1.0 / np.sqrt(((x - m) ** 2).mean(axis=-1, keepdims=True) + eps)
    return (x - m) * r, r


def _each_head(q, k, q_heads, k_heads, d, default):
    q = np.full(d, default) if q is None else q
    k = np.full(d, default) if k is None else k
    return np.stack([q] * q_heads + [k] * k_heads)


def qk_norm(x, q_heads, k_heads, eps, centred, gains=(None, None), shifts=(None, None),
            turn=None):
    """x [tokens, q_heads + k_heads, d]; turn: arguments of attention_opt.rotary
    after x, or None."""
    d = x.shape[-1]
    n, _ = _moments(x, eps, centred)
    y = n * _each_head(*gains, q_heads, k_heads, d, 1.0) + \
        _each_head(*shifts, q_heads, k_heads, d, 0.0)
    return y if turn is None else rotary(y, *turn)


def qk_norm_backward(x, dout, q_heads, k_heads, eps, centred, gains=(None, None), turn=None):
    """dx, and the gradients of the gains and shifts [(q, k), (q, k)]; with each
    the sum of the sizes of its terms."""
    d = x.shape[-1]
    n, r = _moments(x, eps, centred)
    t = dout if turn is None else rotary(dout, *turn, inverse=True)
    u = t * _each_head(*gains, q_heads, k_heads, d, 1.0)
    dx = u - n * (u * n).mean(axis=-1, keepdims=True)
    size = np.abs(u) + np.abs(n) * np.abs(u * n).mean(axis=-1, keepdims=True)
    if centred:
        dx = dx - u.mean(axis=-1, keepdims=True)
        size = size + np.abs(u).mean(axis=-1, keepdims=True)
    cut = (slice(0, q_heads), slice(q_heads, None))
    sums = [[(w[:, c].sum(axis=(0, 1)), np.abs(w[:, c]).sum(axis=(0, 1))) for c in cut]
            for w in (t * n, t)]
    return dx * r, size * r, sums


def default_scale(d):
    return 1.0 / math.sqrt(d)
