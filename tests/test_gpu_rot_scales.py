"""Slab scales that are no scale, on the way of rotated rows: the row's part under that scale is left
out and flagged; its other heads, its other side and its queries are written."""
import numpy as np
import pytest

import cache_testutil as T
import latent_testutil as L
from test_gpu_rot_rows import H, same, to_device  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu
BAD = np.array([np.nan, 0.0, -1.0, np.inf, 2.0 ** -61, 2.0 ** 61], np.float32)


@pytest.mark.parametrize("dtype", ["fp8", "fp4"])
@pytest.mark.parametrize("row,pairs", [("bf16", True), ("f32", False)])
@pytest.mark.parametrize("d,Hkv,Hq,rot,n", [(64, 2, 4, 64, 150), (128, 3, 5, 32, 150), (64, 2, 4, 32, 7200)])
def test_bad_slab_scales(H, dtype, row, pairs, d, Hkv, Hq, rot, n):  # noqa: F811
    """About every third slab of K and of V has one, some pages on both sides (7200 rows: two a warp)."""
    import torch

    rng = np.random.default_rng(61)
    lens, counts = [n + 37, 64], [n, 64]
    rs = T.starts(counts)
    pages = sum(-(-t // 64) for t in lens) + 1
    c = T.make_cache(rng, dtype, pages, Hkv, d)
    bt = T.make_table(rng, lens, pages)
    left_out = {side: rng.random((pages, Hkv)) < 0.35 for side in "kv"}
    left_out["k"][bt[1, 0]] = True  # one page without any K
    good = {**c}
    for side in "kv":
        c[side + "_scale"] = np.where(left_out[side], BAD[rng.integers(0, len(BAD), (pages, Hkv))], c[side + "_scale"])
    x = rng.standard_normal((int(rs[-1]), 2 * Hkv + Hq, d)).astype(np.float32)
    x = x if row == "f32" else T.widen(T.bf16_round(x)).astype(np.float32)
    k, v, q = x[:, :Hkv], x[:, Hkv:2 * Hkv], x[:, 2 * Hkv:]
    table = L.rot_table(max(lens), rot)
    r, pos = L.positions(rs, lens)
    _, pg, ln = T.places(rs, lens, bt)
    want = T.write_rows(good, L.rotate(k[r], pos, table, pairs).astype(np.float64), "k", r, pg, ln)
    want = T.write_rows(want, v.astype(np.float64), "v", r, pg, ln)
    for side in "kv":
        for name in (side, side + "_sf"):
            if name in want:
                want[name][left_out[side]] = c[name][left_out[side]]
    kv = T.device_cache(H, c, bt, lens)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = H.hs2_kv_write_rot(kv, to_device(k, row), to_device(v, row), T.device(rs), T.device(table),
                             style="pairs" if pairs else "halves", q=to_device(q, row), dev_err=err)
    assert int(err.item()) == H.DEV_BAD_PAGE
    arrays = T.cache_arrays(kv, c)
    for name in ("k", "v", "k_sf", "v_sf"):
        if name in arrays:
            assert np.array_equal(arrays[name], want[name]), name
    assert same(T.host(got), T.bf16_round(L.rotate(q[r], pos, table, pairs)))
