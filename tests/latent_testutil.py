"""Plain 64-bit forms of latent attention and of rotated rows."""
from __future__ import annotations

import numpy as np

import cache_testutil as T

PAGE = 64


def rot_table(positions, dim, base=10000.0):
    a = np.arange(positions)[:, None] * base ** (-np.arange(0, dim, 2) / dim)
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def rotate(x, pos, table, pairs):
    """Rows x [n][heads][d] (float32), the first channels rotated, in float32 operation by operation."""
    half = table.shape[1] // 2
    c, s = table[pos][:, None, :half], table[pos][:, None, half:]
    x = x.astype(np.float32).copy()
    ia, ib = (np.arange(0, 2 * half, 2), np.arange(1, 2 * half, 2)) if pairs else (np.arange(half), half + np.arange(half))
    a, b = x[..., ia], x[..., ib]
    with np.errstate(invalid="ignore", over="ignore"):
        x[..., ia], x[..., ib] = a * c - b * s, b * c + a * s
    return x


def positions(rs, lens):
    """(rows, positions) of every row of the batch."""
    r, p = [], []
    for b, t in enumerate(lens):
        n = rs[b + 1] - rs[b]
        r += range(rs[b], rs[b + 1])
        p += range(t - n, t)
    return np.array(r, int), np.array(p, int)


def values(raw):
    return T.widen(raw) if raw.dtype == np.uint16 else raw.astype(np.float64)


def raw(x, dtype):
    return np.ascontiguousarray(x, np.float32) if dtype == "f32" else T.bf16_round(x)


def softmax_rows(x, v):
    """o, lse and sum p |v| / Z of logits x [rows][keys] (-inf: hidden) over values v."""
    m = np.where(np.isfinite(x.max(1, initial=-np.inf)), x.max(1, initial=-np.inf), 0)[:, None]
    p = np.exp(x - m)
    Z = p.sum(1, keepdims=True)
    with np.errstate(divide="ignore", invalid="ignore"):
        return np.where(Z > 0, p @ v / Z, 0), (m + np.log(Z))[:, 0], np.where(Z > 0, p @ np.abs(v) / Z, 0)


def absorbed(pool, q, rs, lens, bt, scale):
    """o, lse, mag of hs2_latent_chunk; pool [pages][64][dc + 64] and q in 64 bits."""
    n, Hq, d = q.shape
    dc = d - 64
    o, lse, mag = np.zeros((n, Hq, dc)), np.full((n, Hq), -np.inf), np.zeros((n, Hq, dc))
    for b, t in enumerate(lens):
        r0, r1 = rs[b], rs[b + 1]
        if r1 <= r0:
            continue
        s = np.arange(t)
        page = bt[b, s // PAGE]
        s = s[(page >= 0) & (page < len(pool))]
        k = pool[bt[b, s // PAGE], s % PAGE]
        seen = s <= (t - (r1 - r0) + np.arange(r1 - r0))[:, None]
        for h in range(Hq):
            x = np.where(seen, scale * q[r0:r1, h] @ k.T, -np.inf)
            o[r0:r1, h], lse[r0:r1, h], mag[r0:r1, h] = softmax_rows(x, k[:, :dc])
    return o, lse, mag


def expanded(q, k, r, v, rs, ks, scale):
    """o, lse, mag of hs2_latent_prefill, all in 64 bits."""
    n, Hq, _ = q.shape
    o, lse, mag = np.zeros((n, Hq, 128)), np.full((n, Hq), -np.inf), np.zeros((n, Hq, 128))
    for b in range(len(rs) - 1):
        r0, r1, k0, k1 = rs[b], rs[b + 1], ks[b], ks[b + 1]
        if r1 <= r0:
            continue
        t = k1 - k0
        seen = np.arange(t) <= (t - (r1 - r0) + np.arange(r1 - r0))[:, None]
        for h in range(Hq):
            x = scale * (q[r0:r1, h, :128] @ k[k0:k1, h].T + q[r0:r1, h, 128:] @ r[k0:k1].T)
            o[r0:r1, h], lse[r0:r1, h], mag[r0:r1, h] = softmax_rows(np.where(seen, x, -np.inf), v[k0:k1, h])
    return o, lse, mag
