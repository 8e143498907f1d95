"""Rotary positions, interval masks and attention over them, in float64 numpy.

Written from the formulas, one head (and, for the masks, one token) at a time,
without the library.  `attention_*` also return how far a bf16 pipeline with
32-bit sums may be off, element by element, counted in half steps of a bf16
rounding (2^-8 of the value): where P and dz become operands of a product, and
where a result is stored.
"""
from __future__ import annotations

import bisect
import math

import numpy as np

HALF_BF16 = 2.0 ** -8     # a rounding to bf16, relative
F32_SLACK = 2.0 ** -16    # 32-bit sums, exponentials and logarithms of a few hundred terms


# ------------------------------------------------------------------ rotary
def axis_of_pair(sections, dealt=False):
    """Axis of each pair: sections in order, or dealt in turn while they last."""
    if not dealt:
        return [x for x, n in enumerate(sections) for _ in range(n)]
    left, out = list(sections), []
    while sum(left):
        for x in range(len(left)):
            if left[x]:
                left[x] -= 1
                out.append(x)
    return out


def rotary(x, positions, inv_freq, rot_dim, sections, adjacent=False, dealt=False, inverse=False):
    """x [tokens, heads, head_dim]; positions [axes, tokens]; inv_freq [rot_dim / 2]."""
    y = np.array(x, dtype=np.float64)
    axes = axis_of_pair(sections, dealt)
    for p in range(rot_dim // 2):
        # whole turns taken off in exact integer arithmetic: inv_freq (a float32
        # value) and the position are rationals, 2 pi to 50 digits
        w = np.array([_reduced(int(t), float(inv_freq[p])) for t in positions[axes[p]]])
        if inverse:
            w = -w
        i, j = (2 * p, 2 * p + 1) if adjacent else (p, p + rot_dim // 2)
        u, v = y[:, :, i].copy(), y[:, :, j].copy()
        y[:, :, i] = u * np.cos(w)[:, None] - v * np.sin(w)[:, None]
        y[:, :, j] = u * np.sin(w)[:, None] + v * np.cos(w)[:, None]
    return y


_TWO_PI = (62831853071795864769252867665590057683943387987502, 10 ** 49)


def _reduced(position, freq):
    """position * freq modulo 2 pi, as a float64."""
    num, den = freq.as_integer_ratio()
    num *= position
    # turns = num / den / (2 pi); what is left of a whole turn, times 2 pi
    big = num * _TWO_PI[1]
    unit = den * _TWO_PI[0]
    rest = big % unit
    if 2 * rest > unit:
        rest -= unit
    return rest / unit * (2 * math.pi)


# ------------------------------------------------------------------ masks
def document_intervals(offsets, prefix, causal, window, b, s):
    """key_lo, key_hi [b, s] of packed documents, token by token."""
    lo, hi = np.zeros((b, s), dtype=np.int64), np.zeros((b, s), dtype=np.int64)
    n = len(offsets) - 1
    for bi in range(b):
        for i in range(s):
            t = bi * s + i
            k = bisect.bisect_right(offsets, t) - 1  # the last document that starts at or before t
            if not 0 <= k < n:
                continue
            pre = prefix[k] if prefix is not None else 0
            if pre < 0:
                continue
            first, last = max(offsets[k], bi * s), min(offsets[k + 1], (bi + 1) * s)
            seen = [j for j in range(first, last)
                    if (not causal or j <= t or j < offsets[k] + pre)
                    and (window == 0 or abs(j - t) < window)]
            lo[bi, i], hi[bi, i] = seen[0] - bi * s, seen[-1] + 1 - bi * s
            assert seen == list(range(seen[0], seen[-1] + 1))
    return lo, hi


def tables(lo, hi, sort=True):
    """The two tables of {sequence, block, first, end}, as lists of tuples."""
    b, s = lo.shape
    nb = (s + 127) // 128
    q, k = [], []
    for bi in range(b):
        union = []
        for blk in range(nb):
            rows = [(int(x), int(y)) for x, y in zip(lo[bi, blk * 128:(blk + 1) * 128],
                                                     hi[bi, blk * 128:(blk + 1) * 128])]
            rows = [(max(x, 0), min(y, s)) for x, y in rows]
            rows = [r for r in rows if r[0] < r[1]]
            union.append((min(r[0] for r in rows), max(r[1] for r in rows)) if rows else (0, 0))
        q += [(bi, blk) + u for blk, u in enumerate(union)]
        for blk in range(nb):
            sees = [x for x, u in enumerate(union)
                    if u[0] < u[1] and u[0] < (blk + 1) * 128 and u[1] > blk * 128]
            k.append((bi, blk) + ((sees[0], sees[-1] + 1) if sees else (0, 0)))
    if sort:
        q.sort(key=lambda e: -(e[3] - e[2]))  # stable
        k.sort(key=lambda e: -(e[3] - e[2]))
    return q, k


# ------------------------------------------------------------------ attention
def _scores(q, k, lo, hi, slope, cap):
    """Scores [s, s] with -inf where masked, and 1 - tanh^2."""
    s, d = q.shape
    z = q @ k.T / math.sqrt(d)
    grad = np.ones_like(z)
    if cap > 0:
        t = np.tanh(z / cap)
        grad = 1.0 - t * t
        z = cap * t
    i, j = np.arange(s)[:, None], np.arange(s)[None, :]
    z = z - slope * np.abs(i - j)
    seen = (j >= lo[:, None]) & (j < hi[:, None])
    return np.where(seen, z, -np.inf), grad, seen


def _softmax(z):
    m = z.max(axis=1, keepdims=True)
    m = np.where(np.isfinite(m), m, 0.0)
    e = np.exp(z - m)
    l = e.sum(axis=1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = (m + np.log(l))[:, 0]
    return e / np.where(l > 0, l, 1.0), lse


def _head(x, n, h, H, d):
    return x[:, n * H * d + h * d: n * H * d + (h + 1) * d]


def attention_forward(qkv, lo, hi, H, d, slopes=None, cap=0.0):
    """qkv [b, s, 3 H d] -> o [b, s, H d], lse [b, H, s], tolerance of o, of lse."""
    b, s, _ = qkv.shape
    o, tol = np.zeros((b, s, H * d)), np.zeros((b, s, H * d))
    lse, ltol = np.zeros((b, H, s)), np.zeros((b, H, s))
    for bi in range(b):
        for h in range(H):
            q, k, v = (_head(qkv[bi], n, h, H, d) for n in range(3))
            z, _, seen = _scores(q, k, lo[bi], hi[bi], 0.0 if slopes is None else slopes[h], cap)
            p, n = _softmax(z)
            cols = slice(h * d, (h + 1) * d)
            o[bi, :, cols], lse[bi, h] = p @ v, n
            # an exponent is off by the 32-bit error of its score
            size = np.where(seen, np.abs(np.where(seen, z, 0.0)), 0.0).max(axis=1) + cap + 1.0
            ltol[bi, h] = F32_SLACK / 8 * size
            mass = p @ np.abs(v)
            tol[bi, :, cols] = (HALF_BF16 + F32_SLACK * size[:, None]) * mass + \
                HALF_BF16 * np.abs(o[bi, :, cols]) + 1e-30
    return o, lse, tol, ltol


def attention_backward(qkv, dout, lo, hi, H, d, slopes=None, cap=0.0):
    """dqkv [b, s, 3 H d], its tolerance, and the part of that which 32-bit
    arithmetic alone may be off (where dP and delta cancel, as in a row that
    sees one key, nothing else is left)."""
    b, s, _ = qkv.shape
    out, tol, tol32 = np.zeros_like(qkv), np.zeros_like(qkv), np.zeros_like(qkv)
    r = 1.0 / math.sqrt(d)
    for bi in range(b):
        for h in range(H):
            q, k, v = (_head(qkv[bi], n, h, H, d) for n in range(3))
            do = _head(dout[bi], 0, h, H, d)
            z, grad, seen = _scores(q, k, lo[bi], hi[bi], 0.0 if slopes is None else slopes[h],
                                    cap)
            p, _ = _softmax(z)
            dp = do @ v.T
            o = p @ v
            delta = (o * do).sum(axis=1, keepdims=True)
            dz = p * (dp - delta) * grad
            size = np.where(seen, np.abs(np.where(seen, z, 0.0)), 0.0).max(axis=1,
                                                                           keepdims=True) + cap + 1.0
            rel = F32_SLACK * size
            # delta is formed from the stored O: one rounding of P and one of O
            ddelta = ((2 * HALF_BF16 + rel) * (p @ np.abs(v)) * np.abs(do)).sum(axis=1,
                                                                                keepdims=True)
            edz32 = p * rel * (np.abs(do) @ np.abs(v).T + np.abs(delta))
            edz = HALF_BF16 * np.abs(dz) + p * grad * ddelta + edz32
            ep = (HALF_BF16 + rel) * p
            for n, (g, e, e32) in enumerate((
                    ((dz @ k) * r, (edz @ np.abs(k)) * r, (edz32 @ np.abs(k)) * r),
                    ((dz.T @ q) * r, (edz.T @ np.abs(q)) * r, (edz32.T @ np.abs(q)) * r),
                    (p.T @ do, ep.T @ np.abs(do), (p * rel).T @ np.abs(do)))):
                cols = slice(n * H * d + h * d, n * H * d + (h + 1) * d)
                out[bi, :, cols] = g
                tol[bi, :, cols] = e * (1 + HALF_BF16) + HALF_BF16 * np.abs(g) + 1e-30
                tol32[bi, :, cols] = e32
    return out, tol, tol32
