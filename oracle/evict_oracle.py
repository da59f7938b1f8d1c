"""fp64 oracle of attention for chunks of new tokens, of the attention weight
that every cached row receives, and of the choice of the rows to keep, in
plain numpy, with the bounds that a computation in 32 bits keeps to."""

from __future__ import annotations

import numpy as np

LATENT = 512


def chunk_visible(n: int, L: int, i: int, causal: bool) -> int:
    """Rows that token i of n sees of L."""
    return max(0, min(L, L - n + i + 1)) if causal else L


def chunk_attend(q, rows, starts, scale: float, causal: bool = True):
    """q [T, H, 576], rows: each request's cached rows [L, 576], starts [B + 1]
    -> out [T, H, 512] (NaN for tokens of no request), lse [T, H]."""
    q, scale = np.asarray(q, np.float64), float(np.float32(scale))  # (the calls take it in 32 bits)
    T, H = q.shape[:2]
    out, lse = np.full((T, H, LATENT), np.nan), np.full((T, H), np.nan)
    for b, row in enumerate(rows):
        n = starts[b + 1] - starts[b]
        for i in range(n):
            t, seen = starts[b] + i, chunk_visible(n, len(row), i, causal)
            out[t], lse[t] = 0.0, -np.inf
            if seen:
                s = scale * (q[t] @ row[:seen].T)
                m = s.max(-1, keepdims=True)
                e = np.exp(s - m)
                z = e.sum(-1, keepdims=True)
                out[t], lse[t] = (e / z) @ row[:seen, :LATENT], (m + np.log(z))[:, 0]
    return out, lse


def score_error(a, s, m):
    """Relative error of exp(score - m) where the score is a sum of 576 bf16
    products in fp32 in any order, a the sum of their magnitudes (scaled): 576
    2^-23 a, the exponent's argument 2^-22 of its size in log2 (1.45 of it), and
    exp2 and one more rounding 2^-21."""
    return 576 * 2.0 ** -23 * a + 2.0 ** -22 * (np.abs(s) + np.abs(m)) * 1.45 + 2.0 ** -21


def chunk_error_bound(q, rows, starts, scale: float, out, causal: bool = True):
    """Bounds (of |out| before its own rounding, of |lse|) on a computation with
    scores and sums in fp32 and softmax weights, values and partial results in
    fp16.

    As for the expanded prefix (prefix_oracle.attend_error_bound): a relative
    error d_j on weight p_j moves the normalised sum by p_j d_j (v_j - out); a
    weight's rounding is 2^-11 of it, or, below fp16's normal range, 2^-25 of a
    weight of one, which the largest is not below.  A value below 2^-14 is off by
    2^-25, a partial result by 2^-11 of itself (at most sum p |v|)."""
    q, scale = np.asarray(q, np.float64), float(np.float32(scale))  # (the calls take it in 32 bits)
    T, H = q.shape[:2]
    bo, bl = np.zeros((T, H, LATENT)), np.zeros((T, H))
    for b, row in enumerate(rows):
        n = starts[b + 1] - starts[b]
        for i in range(n):
            t, seen = starts[b] + i, chunk_visible(n, len(row), i, causal)
            if not seen:
                continue
            k, v = row[:seen], row[:seen, :LATENT]
            s = scale * (q[t] @ k.T)
            a = scale * (np.abs(q[t]) @ np.abs(k).T)
            m = s.max(-1, keepdims=True)
            e = np.exp(s - m)
            z = e.sum(-1, keepdims=True)
            p = e / z
            eta = score_error(a, s, m).max(-1)
            mass = p @ np.abs(v)
            # sum_j p_j |v_j - out|, at most
            spread = np.minimum(mass + np.abs(out[t]), np.sqrt(np.maximum(p @ v ** 2 - out[t] ** 2, 0.0)))
            most = np.abs(v).max(0) + np.abs(out[t])
            bo[t] = ((2.0 ** -11 + 2 * eta[:, None]) * spread * 1.01 + 2.0 ** -25 * (seen / z) * most + 2.0 ** -25
                     + (seen * 2.0 ** -23 + 2.0 ** -11 + 2.0 ** -20) * mass)
            bl[t] = eta + seen * 2.0 ** -24 + 2.0 ** -21 * (1 + np.abs(m[:, 0]) + np.log(z[:, 0]))
    return bo, bl


def attention_weights(q, lse, rows, starts, scale: float, causal: bool = True):
    """What each request's rows received [L], and the bound on it: a relative
    error of score_error (against lse in m's place) on every term, and the sum
    of at most n terms in fp32."""
    q, lse, scale = np.asarray(q, np.float64), np.asarray(lse, np.float64), float(np.float32(scale))
    got, bound = [], []
    for b, row in enumerate(rows):
        n, L = starts[b + 1] - starts[b], len(row)
        w, e = np.zeros(L), np.zeros(L)
        for i in range(n):
            t, seen = starts[b] + i, chunk_visible(n, L, i, causal)
            l = lse[t][:, None]
            s = scale * (q[t] @ row[:seen].T)
            a = scale * (np.abs(q[t]) @ np.abs(row[:seen]).T)
            term = np.where(l == -np.inf, 0.0, np.exp(s - np.where(l == -np.inf, 0.0, l)))
            w[:seen] += term.sum(0)
            e[:seen] += (term * score_error(a, s, np.where(l == -np.inf, 0.0, l))).sum(0)
        got.append(w)
        bound.append(1.01 * e + (128 * n + 2) * 2.0 ** -24 * w)
    return got, bound


def evict_select(weights, L: int, keep: int, sinks: int = 0, recent: int = 0):
    """Positions (increasing) of the rows that stay of one request of L rows."""
    w = np.asarray(weights, np.float64)[:L]
    if L <= keep:
        return np.arange(L)
    w = np.where(np.isnan(w), -np.inf, w)
    fixed = [j for j in range(L) if j < sinks or j >= L - recent]
    rest = sorted((j for j in range(L) if sinks <= j < L - recent), key=lambda j: (-w[j], j))
    return np.array(sorted(fixed + rest[:keep - len(fixed)]))
