"""Plain 64-bit forms of the paged-cache operators, and seeded caches to run them on."""
from __future__ import annotations

import numpy as np

from oracle import hs2_oracle as O

PAGE = 64
E4M3 = O.fp8_e4m3_to_f64(np.arange(127, dtype=np.uint8))  # ascending by code
E2M1 = O.fp4_e2m1_to_f64(np.arange(8, dtype=np.uint8))


def bf16_round(x):
    """float32 to bfloat16 bits, nearest even (NaN kept)."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7FC0), r)


def widen(bits):
    return O.to_f64(bits, "bf16")


def _nearest_code(a, mags):
    """Index of the magnitude nearest to a (inf saturates); the even one on a tie."""
    a = np.minimum(a, mags[-1])
    hi = np.clip(np.searchsorted(mags, a), 1, len(mags) - 1)
    lo = hi - 1
    dl, dh = a - mags[lo], mags[hi] - a
    return np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)


def quantise(x, S, dtype):
    """(codes, group scale codes) of rows x [.., d] (float64 values) with slab scale S [..]."""
    S = np.asarray(S, np.float64)[..., None]
    if dtype == "fp8":
        q = x / S
        code = _nearest_code(np.abs(np.where(np.isnan(q), 0, q)), E4M3)
        code = np.where(np.isnan(x), 0x7F, code)
        return (code | (np.signbit(x) << 7)).astype(np.uint8), None
    g = x.reshape(*x.shape[:-1], -1, 16)
    A = np.abs(g).max(-1)
    nan = np.isnan(A)
    s = np.where(nan, 0x7F, np.minimum(np.searchsorted(6 * E4M3, np.where(nan, 0, A) / S), 126))
    unit = np.where(nan, 0.0, E4M3[np.minimum(s, 126)] * S)[..., None]
    q = np.abs(np.where(np.isnan(g), 0, g)) / np.where(unit > 0, unit, 1)
    code = np.where(unit > 0, _nearest_code(q, E2M1), 0) | (np.signbit(g) << 3)
    code = code.reshape(x.shape).astype(np.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), s.astype(np.uint8)


def make_cache(rng, dtype, num_pages, Hkv, d, scale=1 / 16, key_only=False):
    """A cache's arrays with N(0, 1)-like values in every row."""
    c = {"dtype": dtype, "d": d, "Hkv": Hkv, "num_pages": num_pages}
    for side in ("k",) if key_only else ("k", "v"):
        x = rng.standard_normal((num_pages, Hkv, PAGE, d)).astype(np.float32)
        if dtype == "f32":
            c[side] = x
        elif dtype == "bf16":
            c[side] = bf16_round(x)
        else:
            S = (scale * (0.75 + 0.5 * rng.random((num_pages, Hkv)))).astype(np.float32)
            c[side + "_scale"] = S
            codes, sf = quantise(x.astype(np.float64), np.broadcast_to(S[:, :, None], x.shape[:3]), dtype)
            c[side] = codes
            if sf is not None:
                c[side + "_sf"] = sf
    return c


def values(c, side, page, g, line):
    """float64 values of pool rows (page, g, line) (index arrays)."""
    raw = c[side][page, g, line]
    if c["dtype"] in ("f32", "bf16"):
        return O.to_f64(raw, c["dtype"])
    S = c[side + "_scale"][page, g].astype(np.float64)[..., None]
    if c["dtype"] == "fp8":
        return O.fp8_e4m3_to_f64(raw) * S
    sf = O.fp8_e4m3_to_f64(c[side + "_sf"][page, g, line])
    return O.fp4_e2m1_to_f64(O.fp4_unpack(raw)) * np.repeat(sf, 16, -1) * S


def make_table(rng, lens, num_pages, width=None):
    need = [-(-max(t, 0) // PAGE) for t in lens]
    width = width or max(need + [1])
    order = rng.permutation(num_pages)
    bt = np.full((len(lens), width), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        bt[b, :n] = order[at:at + n]
        at += n
    return bt


def starts(counts, first=0):
    return np.concatenate([[first], first + np.cumsum(counts)]).astype(np.int32)


def places(row_start, lens, bt):
    """(row, page, line) arrays of every row of the batch."""
    r, pg, ln = [], [], []
    for b, t in enumerate(lens):
        n = row_start[b + 1] - row_start[b]
        for i in range(n):
            p = t - n + i
            r.append(row_start[b] + i)
            pg.append(bt[b, p // PAGE])
            ln.append(p % PAGE)
    return np.array(r, int), np.array(pg, int), np.array(ln, int)


def write_rows(c, rows, side, r, pg, ln):
    """The pool arrays after rows[r] (float64 values [n][Hkv][d]) land at (pg, ln)."""
    out = {k: v.copy() if isinstance(v, np.ndarray) else v for k, v in c.items()}
    x = rows[r].astype(np.float64)
    for g in range(c["Hkv"]):
        if c["dtype"] == "f32":
            out[side][pg, g, ln] = x[:, g].astype(np.float32)
        elif c["dtype"] == "bf16":
            out[side][pg, g, ln] = bf16_round(x[:, g].astype(np.float32))
        else:
            codes, sf = quantise(x[:, g], c[side + "_scale"][pg, g], c["dtype"])
            out[side][pg, g, ln] = codes
            if sf is not None:
                out[side + "_sf"][pg, g, ln] = sf
    return out


def attend(c, q, row_start, lens, bt, scale, w=0, sink=None):
    """o, lse of every row in 64 bits, and A = sum p |v| / Z, the scale of o's rounding errors.
    Keys whose page is out of range are left out."""
    n, Hq, d = q.shape
    G = Hq // c["Hkv"]
    o, lse, mag = np.zeros((n, Hq, d)), np.full((n, Hq), -np.inf), np.zeros((n, Hq, d))
    for b, t in enumerate(lens):
        r0, r1 = row_start[b], row_start[b + 1]
        if r1 <= r0:
            continue
        s = np.arange(t)
        page = bt[b, s // PAGE]
        s = s[(page >= 0) & (page < c["num_pages"])]
        page = bt[b, s // PAGE]
        p = t - (r1 - r0) + np.arange(r1 - r0)[:, None]
        seen = (s <= p) & ((s > p - w) if w else True)
        for g in range(c["Hkv"]):
            k, v = (values(c, side, page, g, s % PAGE) for side in ("k", "v"))
            for h in range(g * G, (g + 1) * G):
                x = np.where(seen, scale * q[r0:r1, h].astype(np.float64) @ k.T, -np.inf)
                e = -np.inf if sink is None else float(sink[h])
                m = np.maximum(x.max(1, initial=-np.inf), e)
                m = np.where(np.isfinite(m), m, 0)[:, None]
                pr = np.exp(x - m)
                Z = pr.sum(1, keepdims=True) + np.exp(e - m)
                with np.errstate(divide="ignore", invalid="ignore"):
                    o[r0:r1, h] = np.where(Z > 0, pr @ v / Z, 0)
                    mag[r0:r1, h] = np.where(Z > 0, pr @ np.abs(v) / Z, 0)
                    lse[r0:r1, h] = (m + np.log(Z))[:, 0]
    return o, lse, mag


def device(x):
    import torch

    if x is None:
        return None
    if x.dtype == np.uint16:
        return torch.from_numpy(x.view(np.int16).copy()).cuda().view(torch.bfloat16)
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def host(t):
    import torch

    t = t.detach().cpu()
    return t.view(torch.int16).numpy().view(np.uint16) if t.dtype == torch.bfloat16 else t.numpy()


def device_cache(H, c, bt, lens):
    get = lambda k: device(c.get(k))  # noqa: E731
    return H.KV(k=get("k"), v=get("v"), block_table=device(np.asarray(bt, np.int32)),
                seq_len=device(np.asarray(lens, np.int32)), k_scale=get("k_scale"), v_scale=get("v_scale"),
                k_sf=get("k_sf"), v_sf=get("v_sf"))


def cache_arrays(kv, c):
    return {k: host(getattr(kv, k)) for k in ("k", "v", "k_scale", "v_scale", "k_sf", "v_sf") if k in c}
