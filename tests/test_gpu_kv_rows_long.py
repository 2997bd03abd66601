"""Rows into the cache in calls long enough that a thread takes both K and V of its row, bit for
bit against exact quantisation."""
import numpy as np
import pytest

import cache_testutil as T
from test_gpu_kv_rows import H, check_pools, row_values  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8", "fp4"])
@pytest.mark.parametrize("rows", ["f32", "bf16"])
@pytest.mark.parametrize("d,Hkv,key_only", [(64, 4, False), (128, 2, False), (64, 4, True)])
def test_write_long(H, dtype, rows, d, Hkv, key_only):  # noqa: F811
    rng = np.random.default_rng(51)
    counts = [8200 // Hkv - 1000, 0, 1, 999, 5]
    lens = [counts[0] + 37, 0, 64, 999, 3]  # the last one's rows do not fit its length
    rs = T.starts(counts, first=3)
    n = int(rs[-1]) + 2
    assert n * Hkv >= 8192
    pages = sum(-(-t // 64) for t in lens) + 1
    c = T.make_cache(rng, dtype, pages, Hkv, d, scale=1.0, key_only=key_only)
    bt = T.make_table(rng, lens, pages)
    if dtype in ("fp8", "fp4"):
        c["k_scale"][::3] = 0.5
        c["k_scale"][bt[3, 1], 0] = np.inf  # no scale: K's rows of this slab are left out, V's are written
    dev, val = {}, {}
    good = list(lens)
    good[4], cnt = 0, counts[:4] + [0]
    r, pg, ln = T.places(T.starts(cnt, first=3), good, bt)
    want = c
    for side in ("k",) if key_only else ("k", "v"):
        raw, val[side] = row_values(rng, n, Hkv, d, rows)
        dev[side] = T.device(raw)
        want = T.write_rows(want, val[side], side, r, pg, ln)
    if dtype in ("fp8", "fp4"):
        p = bt[3, 1]
        for name in ("k", "k_sf"):
            if name in want:
                want[name][p, 0] = c[name][p, 0]
    import torch

    kv = T.device_cache(H, c, bt, lens)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    H.hs2_kv_write(kv, dev["k"], dev.get("v"), T.device(rs), dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == H.DEV_BAD_LENGTH | (H.DEV_BAD_PAGE if dtype in ("fp8", "fp4") else 0)
    check_pools(kv, c, want)


@pytest.mark.parametrize("dtype", ["fp8", "fp4"])
@pytest.mark.parametrize("times", [1, 5])
@pytest.mark.parametrize("scales", [(1.0, 0.75), (1 / 3, 1.1), (1 + 2.0 ** -23, 1.25), (2.0 ** -60, 2.0 ** 60)])
def test_every_bfloat16(H, dtype, scales, times):  # noqa: F811
    """Every finite bfloat16 as a row value, in an order where a group's values are neighbours (so that
    they reach all codes) and in one where its largest decides: short quotients, exact and nearly so."""
    import torch

    bits = np.arange(1 << 16, dtype=np.uint16)
    bits = bits[(bits & 0x7F80) != 0x7F80]
    rng = np.random.default_rng(52)
    d, n = 64, times * 2 * len(bits) // 64
    # a group of neighbours in magnitude, both signs; a group within a factor of 16 of its largest
    near = np.concatenate([bits[:len(bits) // 2].reshape(-1, 8), bits[len(bits) // 2:].reshape(-1, 8)], 1).reshape(-1)
    spread = near[:len(bits) // 4096 * 4096].reshape(-1, 256, 16).transpose(0, 2, 1).reshape(-1)
    spread = np.concatenate([spread, rng.permutation(bits)[: len(bits) - len(spread)]])
    raw = np.tile(np.concatenate([near, spread]), times).reshape(n, 1, d)
    val = T.widen(raw)
    pages = -(-n // 64)
    c = T.make_cache(rng, dtype, pages, 1, d)
    c["k_scale"][:], c["v_scale"][:] = scales
    bt = np.arange(pages, dtype=np.int32)[None]
    rs = T.starts([n])
    kv = T.device_cache(H, c, bt, [n])
    r, pg, ln = T.places(rs, [n], bt)
    want = T.write_rows(T.write_rows(c, val, "k", r, pg, ln), val, "v", r, pg, ln)
    rows = T.device(raw)
    H.hs2_kv_write(kv, rows, rows, T.device(rs))
    torch.cuda.synchronize()
    check_pools(kv, c, want)
