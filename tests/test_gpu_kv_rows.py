"""Rows written into a paged cache (quantised to its type) and read back, against the 64-bit
forms: codes and whole pools bit for bit."""
import numpy as np
import pytest

import cache_testutil as T

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def H():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from top_hs2_fa_gb300 import build
    build.build()
    from top_hs2_fa_gb300 import hs2
    hs2.load()
    return hs2


def row_values(rng, n, Hkv, d, dtype):
    """Rows with small and large groups, zeros, exact ties of E2M1 and E4M3, and float64 values of
    what the GPU gets."""
    x = rng.standard_normal((n, Hkv, d)).astype(np.float32)
    x *= np.exp2(rng.integers(-12, 6, (n, Hkv, d // 16, 1))).repeat(16, -1).reshape(n, Hkv, d)
    ties = rng.choice([0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 6, -0.25, -0.75, -2.5, -0.0], (n, Hkv, d))
    x = np.where(rng.random((n, Hkv, 1)) < 0.3, ties, x).astype(np.float32)
    x[rng.random((n, Hkv)) < 0.1] = 0
    bits = T.bf16_round(x) if dtype == "bf16" else None
    return (bits, T.widen(bits)) if dtype == "bf16" else (x, x.astype(np.float64))


def check_pools(kv, c, want):
    got = T.cache_arrays(kv, c)
    for name in got:
        np.testing.assert_array_equal(got[name], want[name], err_msg=name)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8", "fp4"])
@pytest.mark.parametrize("rows", ["f32", "bf16"])
@pytest.mark.parametrize("d,Hkv", [(128, 4), (64, 1)])
def test_write_and_read_ragged(H, dtype, rows, d, Hkv):
    import torch

    rng = np.random.default_rng(11)
    counts, lens = [1, 0, 63, 64, 65, 130, 0, 7, 1], [65, 9, 63, 64, 200, 131, 0, 71, 1]
    rs = T.starts(counts, first=2)  # rows 0, 1 and the last 3 belong to no sequence
    n = int(rs[-1]) + 3
    c = T.make_cache(rng, dtype, 20, Hkv, d, scale=1.0)
    if dtype in ("fp8", "fp4"):  # powers of two too: exact ties
        c["k_scale"][::2] = 0.5
    bt = T.make_table(rng, lens, 20, width=6)
    kv = T.device_cache(H, c, bt, lens)
    dev, val, want = {}, {}, c
    r, pg, ln = T.places(rs, lens, bt)
    for side in ("k", "v"):
        raw, val[side] = row_values(rng, n, Hkv, d, rows)
        wide = torch.zeros((n, Hkv * d + 48), device="cuda", dtype=torch.float32 if rows == "f32" else torch.bfloat16)
        dev[side] = wide[:, 16:16 + Hkv * d].unflatten(1, (Hkv, d))  # a slice of a wider row
        dev[side].copy_(T.device(raw))
        want = T.write_rows(want, val[side], side, r, pg, ln)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    drs = T.device(rs)
    H.hs2_kv_write(kv, dev["k"], dev["v"], drs, dev_err=err)
    for out_dtype in (torch.float32, torch.bfloat16):
        out = tuple(torch.full((n, Hkv, d), 7.0, device="cuda", dtype=out_dtype) for _ in range(2))
        H.hs2_kv_read(kv, drs, n, dtype=out_dtype, out=out, dev_err=err)
        for side, t in zip(("k", "v"), out):
            x = np.full((n, Hkv, d), 7.0)
            for g in range(Hkv):
                x[r, g] = T.values(want, side, pg, g, ln)
            x = x.astype(np.float32)  # one rounding of the product of codes and scales, as the kernel's
            if dtype in ("fp8", "fp4"):
                S = want[side + "_scale"].astype(np.float32)
                for g in range(Hkv):
                    x[r, g] = (T.values(dict(want, **{side + "_scale": np.ones_like(S)}), side, pg, g, ln)
                               .astype(np.float32) * S[pg, g][:, None])
            if out_dtype == torch.bfloat16:
                x = T.widen(T.bf16_round(x))
            np.testing.assert_array_equal(t.float().cpu().numpy(), x)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    check_pools(kv, c, want)


@pytest.mark.parametrize("dtype", ["fp8", "fp4"])
def test_write_special_values(H, dtype):
    """Infinities saturate, a NaN is kept (FP4: its group), denormals and extreme scales."""
    rng = np.random.default_rng(12)
    d, Hkv = 64, 1
    x = rng.standard_normal((70, Hkv, d)).astype(np.float32)
    x[0, 0, 3], x[1, 0, 17], x[2, 0, 20] = np.inf, -np.inf, np.nan
    x[3], x[4] = 1e-42, np.float32(3e38)
    x[5, 0, :16], x[6, 0, 16:32] = -0.0, 1e-30
    x[7:60] *= np.float32(2.0) ** rng.integers(-70, 70, (53, 1, 1))
    c = T.make_cache(rng, dtype, 4, Hkv, d)
    c["k_scale"][:] = np.array([[2.0 ** -60], [2.0 ** 60], [1.1], [0.3]], np.float32)
    c["v_scale"][:] = np.array([[1e-7], [3e9], [2.0 ** -60], [2.0 ** 60]], np.float32)
    lens = [70, 70]
    bt = np.array([[0, 1], [2, 3]], np.int32)
    for b in range(2):
        rs = T.starts([70 if i == b else 0 for i in range(2)])
        kv = T.device_cache(H, c, bt, lens)
        r, pg, ln = T.places(rs, lens, bt)
        want = T.write_rows(T.write_rows(c, x.astype(np.float64), "k", r, pg, ln), x.astype(np.float64), "v", r, pg, ln)
        H.hs2_kv_write(kv, T.device(x), T.device(x), T.device(rs))
        got = T.cache_arrays(kv, c)
        if dtype == "fp8":  # a NaN's sign is not fixed
            for side in ("k", "v"):
                nan = (want[side] & 0x7F) == 0x7F
                np.testing.assert_array_equal((got[side] & 0x7F) == 0x7F, nan)
                got[side][nan] = want[side][nan]
        else:  # a NaN's group: its scale is NaN, its codes are free
            for side in ("k", "v"):
                nan = np.repeat(want[side + "_sf"] == 0x7F, 8, -1)
                got[side][nan] = want[side][nan]
        for name in got:
            np.testing.assert_array_equal(got[name], want[name], err_msg=f"{name} {b}")


def test_write_key_only_single_tokens_equal_append(H):
    """One row per sequence into a key-only bf16 cache: hs2_kv_append's result."""
    import torch

    rng = np.random.default_rng(13)
    lens = [1, 64, 65, 300]
    c = T.make_cache(rng, "bf16", 12, 2, 128, key_only=True)
    bt = T.make_table(rng, lens, 12)
    rows = T.device(T.bf16_round(rng.standard_normal((4, 2, 128)).astype(np.float32)))
    a, b = T.device_cache(H, c, bt, lens), T.device_cache(H, c, bt, lens)
    H.hs2_kv_write(a, rows, None, T.device(T.starts([1] * 4)))
    H.hs2_kv_append([b], [rows])
    assert torch.equal(a.k.view(torch.int16), b.k.view(torch.int16))


def test_write_flags_and_skips(H):
    """Bad lengths, pages and slab scales are flagged; the rows of the others are written, and
    rows of a read stay as they were."""
    import torch

    rng = np.random.default_rng(14)
    lens, counts = [10, 70, 3, 400, 20], [10, 70, 4, 2, 20]
    c = T.make_cache(rng, "fp4", 6, 1, 64, scale=1.0)
    bt = np.array([[0, -1], [1, 6], [2, -1], [3, 3], [4, -1]], np.int32)
    c["k_scale"][0], c["v_scale"][4] = np.nan, -1.0
    rs = T.starts(counts)
    raw, val = row_values(rng, int(rs[-1]), 1, 64, "f32")
    kv = T.device_cache(H, c, bt, lens)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    H.hs2_kv_write(kv, T.device(raw), T.device(raw), T.device(rs), dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == H.DEV_BAD_PAGE | H.DEV_BAD_LENGTH
    row, page, line = (np.array(v) for v in zip(*[(rs[b] + i, bt[b, i // 64], i % 64)
                                                  for b, n in ((0, 10), (1, 64), (4, 20)) for i in range(n)]))
    kk, vv = page != 0, page != 4  # the slabs whose scale is no scale
    want = T.write_rows(c, val, "k", row[kk], page[kk], line[kk])
    want = T.write_rows(want, val, "v", row[vv], page[vv], line[vv])
    check_pools(kv, c, want)
    out = tuple(torch.full((len(raw), 1, 64), 5.0, device="cuda") for _ in range(2))
    err.zero_()
    H.hs2_kv_read(kv, T.device(rs), len(raw), out=out, dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == H.DEV_BAD_PAGE | H.DEV_BAD_LENGTH
    untouched = np.setdiff1d(np.arange(len(raw)), row)
    assert (out[0].cpu().numpy()[untouched] == 5).all() and (out[1].cpu().numpy()[untouched] == 5).all()


def test_empty_calls(H):
    import torch

    rng = np.random.default_rng(15)
    c = T.make_cache(rng, "fp8", 2, 1, 64)
    kv = T.device_cache(H, c, np.array([[0], [1]]), [5, 64])
    none = torch.empty((0, 1, 64), device="cuda")
    H.hs2_kv_write(kv, none, none, T.device(T.starts([0, 0])))
    k, v = H.hs2_kv_read(kv, T.device(T.starts([0, 0])), 0)
    assert k.shape == (0, 1, 64) and v.shape == (0, 1, 64)
    check_pools(kv, c, c)
