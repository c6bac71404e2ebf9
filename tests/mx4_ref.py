"""The microscaled 4-bit format, its products and the balance loss in float64 (NumPy), from their definitions."""
from __future__ import annotations

import numpy as np

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def quantize(x: np.ndarray):
    """x [..., K] (float32 values) -> codes uint8 [..., 16 B], scales uint8 [..., B]."""
    x = np.asarray(x, np.float64)
    K = x.shape[-1]
    B = -(-K // 32)
    v = np.zeros((*x.shape[:-1], 32 * B))
    v[..., :K] = x
    v = v.reshape(*x.shape[:-1], B, 32)
    top = np.abs(v).max(-1)
    good = np.isfinite(top)
    some = good & (top > 0)
    e = np.full(top.shape, -127)
    e[some] = np.maximum(np.frexp(top[some])[1] - 3, -127)
    m = np.where(good[..., None], np.abs(np.where(np.isfinite(v), v, 0.0)), 0) / 2.0 ** e[..., None]
    mid = (GRID[1:] + GRID[:-1]) / 2   # the borders between neighbours
    code = np.zeros(m.shape, np.uint8)
    for i, b in enumerate(mid):        # past the border, or on it where the upper code is the even one
        code += (m > b) | ((m == b) & (i % 2 == 1))
    code += 8 * (np.signbit(v) & good[..., None]).astype(np.uint8)
    code = code.reshape(*x.shape[:-1], 32 * B)
    scales = np.where(good, e + 127, 255).astype(np.uint8)
    return (code[..., 0::2] | code[..., 1::2] << 4).astype(np.uint8), scales


def values(codes: np.ndarray, scales: np.ndarray, K: int) -> np.ndarray:
    code = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    v = np.concatenate([GRID, -GRID])[code]
    s = np.repeat(np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127)), 32, -1)
    return (v * s)[..., :K]


def token_rows(perm: np.ndarray, T: int, k: int) -> np.ndarray:
    return np.where(perm < T * k, perm // k, perm - T * k)


def grouped(x: np.ndarray, w: np.ndarray, offsets: np.ndarray):
    """Rows x [A, K] of the groups times w [E_tot, N, K]: y [A, N] and sum |x w|; zeros in rows of no group."""
    y = np.zeros((x.shape[0], w.shape[1]))
    size = np.zeros_like(y)
    for e in range(w.shape[0]):
        a, b = offsets[e], offsets[e + 1]
        y[a:b] = x[a:b] @ w[e].T
        size[a:b] = np.abs(x[a:b]) @ np.abs(w[e]).T
    return y, size


def balance(logits: np.ndarray, idx: np.ndarray, keep: np.ndarray, d=None):
    """(losses [2], counts, n, dlogits or None, p, lse)."""
    x = np.asarray(logits, np.float64)
    T, E = x.shape
    k = idx.shape[1]
    n = int(keep.sum())
    ids = idx[keep].ravel()
    counts = np.bincount(ids[(ids >= 0) & (ids < E)], minlength=E)
    top = x.max(1, initial=-np.inf)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        ex = np.where(np.isneginf(top)[:, None], 0.0, np.exp(x - top[:, None]))
        total = ex.sum(1)
        p = np.where(total[:, None] == 0, 0.0, ex / total[:, None])
        lse = np.where(total == 0, 0.0, top + np.log(total))
    if n == 0:
        return np.zeros(2), counts, 0, np.zeros_like(x), p, lse
    f = counts / (n * k)
    losses = np.array([E * (f * p[keep].sum(0) / n).sum(), (lse[keep] ** 2).sum() / n])
    dx = None
    if d is not None:
        dot = p @ f
        dx = p * (d[0] * E / n * (f - dot[:, None]) + d[1] * 2 / n * lse[:, None])
        dx[~keep] = 0
    return losses, counts, n, dx, p, lse
