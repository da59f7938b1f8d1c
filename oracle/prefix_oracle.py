"""fp64 oracle of the expanded shared prefix and of attention over it, in
plain numpy, with the magnitudes that error bounds need."""

from __future__ import annotations

import numpy as np


def prefix_expand(latent, w):
    """latent [P, 512], w [H, 512, 128] -> [H, P, 128]."""
    return np.einsum("pc,hcd->hpd", np.asarray(latent, np.float64), np.asarray(w, np.float64))


def prefix_attend(q_nope, q_pe, k_nope, k_pe, v, scale: float, visible=None, suffix_out=None, suffix_lse=None):
    """q_nope [T, H, 128], q_pe [T, H, 64], k_nope, v [H, P, 128], k_pe [P, 64]
    -> out [T, H, 128], lse [T, H]: token t attends to rows 0 .. visible[t] - 1,
    joined with a suffix's result where given."""
    q_nope, q_pe, k_nope, k_pe, v = (np.asarray(a, np.float64) for a in (q_nope, q_pe, k_nope, k_pe, v))
    T, H = q_nope.shape[:2]
    P = k_nope.shape[1]
    out, lse = np.zeros((T, H, 128)), np.full((T, H), -np.inf)
    for t in range(T):
        n = P if visible is None else int(min(max(visible[t], 0), P))
        if n == 0:
            continue
        s = scale * (np.einsum("hd,hpd->hp", q_nope[t], k_nope[:, :n]) + q_pe[t] @ k_pe[:n].T)
        m = s.max(-1, keepdims=True)
        e = np.exp(s - m)
        z = e.sum(-1, keepdims=True)
        out[t] = np.einsum("hp,hpd->hd", e / z, v[:, :n])
        lse[t] = (m + np.log(z))[:, 0]
    if suffix_out is not None:
        out, lse = join(out, lse, suffix_out, suffix_lse)
    return out, lse


def join(out_a, lse_a, out_b, lse_b):
    """Two attention results over disjoint rows as one over both."""
    lse_a, lse_b = np.asarray(lse_a, np.float64), np.asarray(lse_b, np.float64)
    m = np.maximum(lse_a, lse_b)
    some = np.isfinite(m)
    base = np.where(some, m, 0.0)
    wa, wb = np.exp(lse_a - base), np.exp(lse_b - base)
    z = np.where(some, wa + wb, 1.0)
    a = np.where(wa[..., None] > 0, np.asarray(out_a, np.float64), 0.0) * (wa / z)[..., None]
    b = np.where(wb[..., None] > 0, np.asarray(out_b, np.float64), 0.0) * (wb / z)[..., None]
    return a + b, np.where(some, m + np.log(z), -np.inf)


def attend_error_bound(q_nope, q_pe, k_nope, k_pe, v, scale: float, out, visible=None):
    """Bounds (of |out| before its own rounding [T, H, 128], of |lse| [T, H])
    on a computation that sums bf16 / fp16 products in fp32, takes exp in fp32
    and rounds the weights to fp16, normalising by the rounded sum.

    With p_j the exact weights (sum 1), a score is off by at most 192 * 2^-23 *
    scale * sum_d |q_d k_d| (any order of 192 fp32 additions), its exponent's
    argument by another 2^-22 of its size, exp2 by 2^-21: together eta, relative
    on every weight.  Rounding a weight to fp16 is off by 2^-11 of it or, below
    fp16's normal range, by 2^-25 where the largest weight is at least 1, that
    is 2^-25 / z as a share of the sum z >= 1.  A relative error d_j on weight j
    moves a normalised sum by p_j d_j (v_j - out).  The value sum itself adds n
    2^-23 of sum p |v|, partial results joined in fp32 2^-20 of it."""
    q_nope, q_pe, k_nope, k_pe, v = (np.asarray(a, np.float64) for a in (q_nope, q_pe, k_nope, k_pe, v))
    T, H = q_nope.shape[:2]
    P = k_nope.shape[1]
    bo, bl = np.zeros((T, H, 128)), np.zeros((T, H))
    for t in range(T):
        n = P if visible is None else int(min(max(visible[t], 0), P))
        if n == 0:
            continue
        s = scale * (np.einsum("hd,hpd->hp", q_nope[t], k_nope[:, :n]) + q_pe[t] @ k_pe[:n].T)
        a = scale * (np.einsum("hd,hpd->hp", np.abs(q_nope[t]), np.abs(k_nope[:, :n])) + np.abs(q_pe[t]) @ np.abs(k_pe[:n]).T)
        m = s.max(-1, keepdims=True)
        e = np.exp(s - m)
        z = e.sum(-1, keepdims=True)
        p = e / z
        eta = (192 * 2.0 ** -23 * a + 2.0 ** -22 * (np.abs(s) + np.abs(m)) * 1.45 + 2.0 ** -21).max(-1)
        dev = np.abs(v[:, :n] - out[t][:, None])
        spread = np.einsum("hp,hpd->hd", p, dev)
        mass = np.einsum("hp,hpd->hd", p, np.abs(v[:, :n]))
        bo[t] = (2.0 ** -11 + 2 * eta[:, None]) * spread * 1.01 + 2.0 ** -25 / z * dev.sum(1) + (n * 2.0 ** -23 + 2.0 ** -20) * mass
        bl[t] = eta + n * 2.0 ** -24 + 2.0 ** -21 * (1 + np.abs(m[:, 0]) + np.log(z[:, 0]))
    return bo, bl
