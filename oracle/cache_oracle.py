"""fp64 oracle of rotary positions and of the append to the paged latent cache
(bf16 or FP8 rows), in plain numpy."""

from __future__ import annotations

import numpy as np

D_C, D_R, PAGE, FP8_ROW = 512, 64, 64, 656


def rotate(x, positions, inv_freq, half: bool = False, inverse: bool = False, scale: float = 1.0):
    """x [T, ..., R] float64: pair i of row t turned by positions[t] *
    inv_freq[i] radians (turned back with `inverse`) and scaled."""
    x = np.asarray(x, np.float64)
    R = x.shape[-1]
    ang = np.asarray(positions, np.float64).reshape((-1,) + (1,) * (x.ndim - 1)) * np.asarray(inv_freq, np.float64)
    if inverse:
        ang = -ang
    c, s = np.cos(ang) * scale, np.sin(ang) * scale
    first, second = (slice(0, R // 2), slice(R // 2, R)) if half else (slice(0, R, 2), slice(1, R, 2))
    out = np.empty_like(x)
    out[..., first] = x[..., first] * c - x[..., second] * s
    out[..., second] = x[..., first] * s + x[..., second] * c
    return out


def rope(x, positions, inv_freq, offset: int = 0, half: bool = False, inverse: bool = False, scale: float = 1.0):
    """rotate() of dims [offset, offset + R) of x [T, H, D], the others unchanged."""
    out = np.array(x, np.float64)
    r = slice(offset, offset + 2 * len(inv_freq))
    out[..., r] = rotate(out[..., r], positions, inv_freq, half, inverse, scale)
    return out


def rms_norm(x, weight, eps: float):
    x = np.asarray(x, np.float64)
    return x * np.asarray(weight, np.float64) / np.sqrt((x * x).mean(-1, keepdims=True) + eps)


def group_scales(latent):
    """latent [T, 512]: per group of 128 dims the exponent e of its scale 2^e,
    the smallest with max|x| <= 448 * 2^e (0 for a group of zeros, at least
    -127), over the finite dims.  Returns int [T, 4]."""
    g = np.abs(np.asarray(latent, np.float64).reshape(-1, 4, 128))
    m = np.where(np.isfinite(g), g, 0.0).max(-1)
    e = np.full(m.shape, 0, np.int64)
    nz = m > 0
    e[nz] = np.ceil(np.log2(m[nz] / 448.0)).astype(np.int64)
    # log2 is rounded: settle the exact condition
    e = np.where(nz & (m > 448.0 * 2.0 ** e), e + 1, e)
    e = np.where(nz & (m <= 448.0 * 2.0 ** (e - 1)), e - 1, e)
    return np.maximum(e, -127)


def appended_rows(latent, k_pe, positions, weight=None, eps: float = 1e-6, inv_freq=None, half: bool = False,
                  scale: float = 1.0):
    """The (latent [T, 512], RoPE dims [T, 64]) an append stores, before rounding."""
    lat = np.asarray(latent, np.float64)
    if weight is not None:
        lat = rms_norm(lat, weight, eps)
    pe = np.asarray(k_pe, np.float64)
    if inv_freq is not None:
        pe = rotate(pe, positions, inv_freq, half, False, scale)
    return lat, pe


def append_places(positions, request_ids, block_table):
    """Pool row of each token (-1 for padding)."""
    pos, req, bt = np.asarray(positions), np.asarray(request_ids), np.asarray(block_table)
    rows = np.full(pos.shape, -1, np.int64)
    for t in np.nonzero(pos >= 0)[0]:
        rows[t] = int(bt[req[t], pos[t] // PAGE]) * PAGE + pos[t] % PAGE
    return rows
