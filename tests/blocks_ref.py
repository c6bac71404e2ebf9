"""8-bit blocks and their products, the RMS norm and routing by scores in float64 (NumPy), from their definitions."""
from __future__ import annotations

import numpy as np

LEAST = 2.0 ** -116
_C = np.arange(256)
_E, _M = (_C >> 3) & 15, _C & 7
CODES = np.where(_E == 0, _M / 8 * 2.0 ** -6, (1 + _M / 8) * 2.0 ** (_E - 7.0)) * np.where(_C >= 128, -1, 1)
CODES[[127, 255]] = np.nan
GRID = CODES[:127]
_MID = (GRID[1:] + GRID[:-1]) / 2


def nearest(m: np.ndarray) -> np.ndarray:
    """Codes 0 .. 126 of magnitudes: the nearest, a tie to the even one, past 448 to 448."""
    lo = np.searchsorted(_MID, m, side="left")    # borders below m
    hi = np.searchsorted(_MID, m, side="right")   # borders at or below m
    return np.where((hi > lo) & (lo % 2 == 1), hi, lo).astype(np.uint8)


def quantize(x: np.ndarray, block_rows: int = 1):
    """x [..., R, K] (float32 values) -> codes uint8 [..., R, 128 B], scales float32 [..., ceil(R / block_rows), B]."""
    x = np.asarray(x, np.float64)
    R, K = x.shape[-2:]
    B, G = -(-K // 128), -(-R // block_rows)
    v = np.zeros((*x.shape[:-2], G * block_rows, 128 * B))
    v[..., :R, :K] = x
    b = v.reshape(*x.shape[:-2], G, block_rows, B, 128)
    top = np.abs(b).max((-3, -1))
    good = np.isfinite(top)
    scale = (np.maximum(np.where(good, top, 1), LEAST).astype(np.float32) / np.float32(448)).astype(np.float32)
    full = np.broadcast_to(scale.astype(np.float64)[..., :, None, :, None], b.shape)
    ok = np.broadcast_to(good[..., :, None, :, None], b.shape)
    code = nearest(np.abs(np.where(ok, b, 0)) / full) + 128 * (np.signbit(b) & ok).astype(np.uint8)
    code = code.reshape(v.shape)[..., :R, :].astype(np.uint8)
    return code, np.where(good, scale, np.float32(np.nan)).astype(np.float32)


def values(codes: np.ndarray, scales: np.ndarray, K: int, block_rows: int = 1) -> np.ndarray:
    s = np.repeat(np.asarray(scales, np.float64), 128, -1)
    if block_rows > 1:
        s = np.repeat(s, block_rows, -2)[..., : codes.shape[-2], :]
    return (CODES[codes] * s)[..., :K]


def products(x: np.ndarray, w: np.ndarray):
    """y = x w^T and sum |x w|."""
    return x @ w.T, np.abs(x) @ np.abs(w).T


def cut(x: np.ndarray, w: np.ndarray) -> np.ndarray:
    """What the 8-bit matrix cores may drop of x [T, K] w [N, K]^T: of each of a block's products less than 2^-12 of the
    block's largest (13 bits under the binade of the largest pair of codes, whose product may reach the next one)."""
    T, K = x.shape
    lost = np.zeros((T, w.shape[0]))
    for b in range(0, K, 128):
        a, c = np.abs(x[:, None, b:b + 128]), np.abs(w[None, :, b:b + 128])
        p = a * c
        lost += 2.0 ** -12 * p.max(2) * (p > 0).sum(2)
    return lost


# ---- norm -------------------------------------------------------------------------------


def norm(r: np.ndarray, w: np.ndarray, eps: float) -> np.ndarray:
    return w * r / np.sqrt((r * r).mean(1, keepdims=True) + eps)


def norm_gradients(dy, h, w, d_total, eps):
    """(dh, dweight, and the sums of the magnitudes that each adds up)."""
    q = 1 / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    a = w * dy
    d = 0 if d_total is None else d_total
    dh = d + q * (a - h * q * q * (a * h).mean(1, keepdims=True))
    size = np.abs(d) + q * (np.abs(a) + np.abs(h) * q * q * np.abs(a * h).mean(1, keepdims=True))
    return dh, (dy * h * q).sum(0), size, np.abs(dy * h * q).sum(0)


# ---- routing ----------------------------------------------------------------------------


def scores(logits: np.ndarray, kind: str) -> np.ndarray:
    x = np.asarray(logits, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if kind == "sigmoid":
            return 1 / (1 + np.exp(-x))
        top = x.max(1, keepdims=True)
        ex = np.where(np.isneginf(top), 0.0, np.exp(x - np.where(np.isneginf(top), 0, top)))
        total = ex.sum(1, keepdims=True)
        return np.where(total == 0, 0.0, ex / np.where(total == 0, 1, total))


def route(logits, k, bias=None, score="sigmoid", groups=1, keep_groups=1, group_top=2, renormalize=True, scale=1.0):
    """(idx [T, k], gates [T, k]), token by token."""
    T, E = logits.shape
    s = scores(logits, score)
    size = E // groups
    idx = np.zeros((T, k), np.int32)
    gates = np.zeros((T, k))
    for t in range(T):
        c = s[t] + bias if bias is not None else np.asarray(logits[t], np.float64)
        c = np.where(np.isneginf(logits[t]), -np.inf, c)
        full = s[t] + bias if bias is not None else s[t]
        rank = [(2, 0.0) if np.isnan(v) else (1, 0.0) if np.isneginf(v) else (0, -v) for v in c]
        allowed = range(E)
        if groups > 1:
            worth = []
            for g in range(groups):
                live = sorted((e for e in range(g * size, (g + 1) * size) if rank[e][0] == 0), key=lambda e: (rank[e], e))[:group_top]
                worth.append((0, -sum(full[e] for e in live) if group_top == 2 else rank[live[0]][1], g) if live else (1, 0.0, g))
            kept = {g for _, _, g in sorted(worth)[:keep_groups]}
            allowed = [e for e in range(E) if e // size in kept]
        order = sorted(allowed, key=lambda e: (rank[e], e))[:k]
        idx[t] = order
        q = s[t][order]
        total = q.sum()
        gates[t] = np.float64(np.float32(scale)) * (q if not renormalize else q / total if total != 0 else 0 * q)
    return idx, gates


def route_gradient(logits, idx, d_gates, score="sigmoid", renormalize=True, scale=1.0):
    """(dlogits [T, E], the magnitudes that each adds up)."""
    T, E = logits.shape
    s = scores(logits, score)
    out, size = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        there = (idx[t] >= 0) & (idx[t] < E)
        e = idx[t][there]
        d = np.float64(np.float32(scale)) * d_gates[t][there]
        q = s[t][e]
        m = np.abs(d)
        if renormalize:
            total = q.sum()
            d, m = ((d - (d * q).sum() / total) / total, (m + (m * q).sum() / total) / total) if total != 0 else (0 * d, 0 * m)
        ds, dm = np.zeros(E), np.zeros(E)
        np.add.at(ds, e, d)
        np.add.at(dm, e, m)
        if score == "sigmoid":
            out[t], size[t] = ds * s[t] * (1 - s[t]), dm * s[t]
        else:
            out[t], size[t] = s[t] * (ds - (d * q).sum()), s[t] * (dm + (m * q).sum())
    return out, size
