"""Rows that are rotated on their way into a cache: bit for bit what float32 operations one after
another give, quantised as exact arithmetic has it."""
import numpy as np
import pytest

import cache_testutil as T
import latent_testutil as L

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


def same(a, b):
    """Equal bit for bit, any NaN like any other."""
    if a.dtype == np.uint16:
        a, b = T.widen(a), T.widen(b)
    return a.shape == b.shape and bool((np.equal(a, b) & (np.signbit(a) == np.signbit(b)) | ((a != a) & (b != b))).all())


def rows_of(rng, n, heads, d, row):
    x = (rng.standard_normal((n, heads, d)) * np.exp(rng.standard_normal((n, heads, 1)))).astype(np.float32)
    return x if row == "f32" else T.widen(T.bf16_round(x)).astype(np.float32)


def to_device(x, row):
    return T.device(x if row == "f32" else T.bf16_round(x))


CASES = [(d, Hkv, Hq, rot, pairs) for d, Hkv, Hq in ((64, 1, 0), (64, 3, 5), (128, 1, 8), (128, 4, 32), (128, 2, 3))
         for rot, pairs in ((32, False), (d, False), (d, True), (32, True), (96, False)) if rot <= d]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8", "fp4"])
@pytest.mark.parametrize("row", ["f32", "bf16"])
@pytest.mark.parametrize("d,Hkv,Hq,rot,pairs", CASES)
def test_write(H, dtype, row, d, Hkv, Hq, rot, pairs):
    import torch

    rng = np.random.default_rng(51)
    lens, counts = [5, 200, 64, 1, 0, 130], [5, 3, 64, 1, 0, 1]
    rs = T.starts(counts, 1)
    pages = sum(-(-t // 64) for t in lens) + 1
    c = T.make_cache(rng, dtype, pages, Hkv, d)
    bt = T.make_table(rng, lens, pages)
    n = int(rs[-1]) + 2
    k, v, q = (rows_of(rng, n, h, d, row) for h in (Hkv, Hkv, max(Hq, 1)))
    table = L.rot_table(200, rot)
    r, pos = L.positions(rs, lens)
    turned = k.copy()
    turned[r] = L.rotate(k[r], pos, table, pairs)
    _, pg, ln = T.places(rs, lens, bt)
    want = T.write_rows(T.write_rows(c, turned.astype(np.float64), "k", r, pg, ln), v.astype(np.float64), "v", r, pg, ln)
    kv = T.device_cache(H, c, bt, lens)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out_type = torch.float32 if dtype == "f32" else torch.bfloat16
    q_out = torch.full((n, Hq, d), 9.0, dtype=out_type, device="cuda") if Hq else None
    got = H.hs2_kv_write_rot(kv, to_device(k, row), to_device(v, row), T.device(rs), T.device(table),
                             style="pairs" if pairs else "halves", q=to_device(q, row) if Hq else None, q_out=q_out,
                             dev_err=err)
    assert int(err.item()) == 0
    for name, a in T.cache_arrays(kv, c).items():
        assert np.array_equal(a, want[name]), name
    if Hq:
        wq = np.full((n, Hq, d), 9.0, np.float32)
        wq[r] = L.rotate(q[r], pos, table, pairs)
        assert same(T.host(got), wq if dtype == "f32" else T.bf16_round(wq))


@pytest.mark.parametrize("dtype,row", [("fp4", "bf16"), ("fp8", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("n", [4096, 6999, 7000, 7003, 9001])
def test_many_rows(H, dtype, row, n):
    """About the border where a warp takes several rows, page-unaligned, key and query of their own strides."""
    import torch

    rng = np.random.default_rng(52)
    Hkv, Hq, d, rot = 2, 4, 128, 128
    lens, counts = [n // 2 + 70, n], [n // 2, n - n // 2]
    rs = T.starts(counts)
    pages = sum(-(-t // 64) for t in lens)
    c = T.make_cache(rng, dtype, pages, Hkv, d)
    bt = T.make_table(rng, lens, pages)
    x = rows_of(rng, n, Hq + 2 * Hkv, d, row)
    table = L.rot_table(max(lens), rot)
    r, pos = L.positions(rs, lens)
    _, pg, ln = T.places(rs, lens, bt)
    k = L.rotate(x[:, Hq:Hq + Hkv][r], pos, table, False)
    want = T.write_rows(T.write_rows(c, k.astype(np.float64), "k", r, pg, ln), x[:, Hq + Hkv:].astype(np.float64), "v", r, pg, ln)
    kv = T.device_cache(H, c, bt, lens)
    dx = to_device(x, row)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    v = dx[:, Hq + Hkv:].contiguous()  # another stride than K's
    got = H.hs2_kv_write_rot(kv, dx[:, Hq:Hq + Hkv], v, T.device(rs), T.device(table), q=dx[:, :Hq], dev_err=err)
    assert int(err.item()) == 0
    for name, a in T.cache_arrays(kv, c).items():
        assert np.array_equal(a, want[name]), name
    assert same(T.host(got), T.bf16_round(L.rotate(x[:, :Hq][r], pos, table, False)))


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("row,dtype", [("bf16", "fp8"), ("f32", "f32")])
def test_in_place_and_key_only(H, row, dtype, pairs):
    import torch

    rng = np.random.default_rng(53)
    lens, counts = [70, 500], [2, 300]
    rs = T.starts(counts)
    pages = 11
    c = T.make_cache(rng, dtype, pages, 2, 128, key_only=True)
    bt = T.make_table(rng, lens, pages)
    k, q = rows_of(rng, 302, 2, 128, row), rows_of(rng, 302, 8, 128, row)
    table = L.rot_table(500, 128)
    r, pos = L.positions(rs, lens)
    _, pg, ln = T.places(rs, lens, bt)
    want = T.write_rows(c, L.rotate(k[r], pos, table, pairs).astype(np.float64), "k", r, pg, ln)
    get = lambda s: T.device(c.get(s))  # noqa: E731
    kv = H.KV(k=get("k"), v=None, block_table=T.device(bt), seq_len=T.device(np.array(lens, np.int32)), k_scale=get("k_scale"))
    dq = to_device(q, row)
    got = H.hs2_kv_write_rot(kv, to_device(k, row), None, T.device(rs), T.device(table), style="pairs" if pairs else "halves",
                             q=dq, q_out=dq)
    assert got is dq
    w = L.rotate(q[r], pos, table, pairs)
    assert same(T.host(dq), w if row == "f32" else T.bf16_round(w))
    assert np.array_equal(T.host(kv.k), want["k"])


def test_infinities_and_nan(H):
    """V is not rotated; what is not rotated of K passes; inf and NaN go where the formula takes them."""
    rng = np.random.default_rng(54)
    k, v, q = (rows_of(rng, 3, 1, 64, "f32") for _ in range(3))
    k[0, 0, 3], k[1, 0, 40], v[0, 0, 5], q[2, 0, 17], k[2, 0, 33] = np.inf, np.nan, -np.inf, np.nan, -np.inf
    table = L.rot_table(10, 32)
    table[9, 1] = np.inf
    c = T.make_cache(rng, "f32", 1, 1, 64)
    kv = T.device_cache(H, c, np.zeros((1, 1), np.int32), [10])
    got = H.hs2_kv_write_rot(kv, T.device(k), T.device(v), T.device(T.starts([3])), T.device(table), q=T.device(q))
    pos = np.array([7, 8, 9])
    assert same(T.host(kv.k)[0, 0, 7:10], L.rotate(k, pos, table, False)[:, 0])
    assert same(T.host(kv.v)[0, 0, 7:10], v[:, 0])
    assert same(T.host(got), L.rotate(q, pos, table, False))


def test_flagged_rows(H):
    import torch

    rng = np.random.default_rng(55)
    lens, counts = [100, 200, 130, 3], [4, 2, 3, 5]
    rs = T.starts(counts)
    n = int(rs[-1])
    c = T.make_cache(rng, "bf16", 12, 2, 64)
    bt = T.make_table(rng, lens, 12)
    bt[2, 2] = 12
    table = L.rot_table(198 + 1, 64)  # position 199 has no angles
    k, v, q = (rows_of(rng, n, h, 64, "bf16") for h in (2, 2, 4))
    kv = T.device_cache(H, c, bt, lens)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = torch.full((n, 4, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    H.hs2_kv_write_rot(kv, to_device(k, "bf16"), to_device(v, "bf16"), T.device(rs), T.device(table), q=to_device(q, "bf16"),
                       q_out=q_out, dev_err=err)
    assert int(err.item()) == H.DEV_BAD_LENGTH | H.DEV_BAD_INDEX | H.DEV_BAD_PAGE
    good = [0, 1, 2, 3, 4, 6]  # not: position 199, sequence 2's rows of page 2, sequence 3's
    pos = np.array([96, 97, 98, 99, 198, 127])
    seq = [0, 0, 0, 0, 1, 2]
    pg = bt[seq, pos // 64]
    want = T.write_rows(c, L.rotate(k[good], pos, table, False).astype(np.float64), "k", np.arange(6), pg, pos % 64)
    want = T.write_rows(want, v[good].astype(np.float64), "v", np.arange(6), pg, pos % 64)
    for name, a in T.cache_arrays(kv, c).items():
        assert np.array_equal(a, want[name]), name
    wq = np.full((n, 4, 64), 9.0, np.float32)
    wq[good] = L.rotate(q[good], pos, table, False)
    assert same(T.host(q_out), T.bf16_round(wq))
    rs_bad = rs.copy()
    rs_bad[-1] = n + 3  # rows that do not exist
    err.zero_()
    H.hs2_kv_write_rot(kv, to_device(k, "bf16"), to_device(v, "bf16"), T.device(rs_bad), T.device(table), dev_err=err)
    assert int(err.item()) & H.DEV_BAD_LENGTH


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("row", ["f32", "bf16"])
@pytest.mark.parametrize("dc,Hq,pairs,n1", [(512, 16, True, 3), (256, 1, False, 3), (512, 0, True, 3), (512, 9, False, 3),
                                            (256, 128, True, 70), (512, 2, True, 4300), (512, 9, True, 7103), (256, 0, False, 14100)])
def test_latent_rows(H, dtype, row, dc, Hq, pairs, n1):
    import torch

    rng = np.random.default_rng(56)
    lens, counts = [5, n1 + 100, 64, 0, 130], [5, n1, 64, 0, 1]
    rs = T.starts(counts, 2)
    n = int(rs[-1]) + 1
    pages = sum(-(-t // 64) for t in lens) + 1
    pool = L.raw(rng.standard_normal((pages, 64, dc + 64)), dtype)
    bt = T.make_table(rng, lens, pages)
    x = rows_of(rng, n, 1, dc + 64, row)[:, 0]  # c and r as slices of one projection
    q = rows_of(rng, n, max(Hq, 1), 192, row)
    table = L.rot_table(max(lens), 64)
    r, pos = L.positions(rs, lens)
    _, pg, ln = T.places(rs, lens, bt)
    turned = L.rotate(x[r, None, dc:], pos, table, pairs)[:, 0]
    want = pool.copy()
    want[pg, ln] = L.raw(np.concatenate([x[r, :dc], turned], 1), dtype)
    kv = H.KV(k=T.device(pool[:, None]), v=None, block_table=T.device(bt), seq_len=T.device(np.array(lens, np.int32)))
    dx, dq = to_device(x, row), to_device(q, row)
    out = torch.full((n, max(Hq, 1), dc + 64), 9.0, dtype=torch.float32 if dtype == "f32" else torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    H.hs2_latent_write(kv, dx[:, :dc], dx[:, dc:], T.device(rs), T.device(table), style="pairs" if pairs else "halves",
                       q=dq[..., 128:] if Hq else None, q_out=out[..., dc:] if Hq else None, dev_err=err)
    assert int(err.item()) == 0
    assert np.array_equal(T.host(kv.k)[:, 0], want)
    if Hq:
        w = np.full((n, Hq, dc + 64), 9.0, np.float32)
        w[r, :, dc:] = L.rotate(q[r, :, 128:], pos, table, pairs)
        assert same(T.host(out), L.raw(w, dtype))
    for to in (torch.float32, torch.bfloat16):
        got = torch.full((n, dc), 9.0, dtype=to, device="cuda"), torch.full((n, 72), 9.0, dtype=to, device="cuda")
        H.hs2_latent_read(kv, T.device(rs), n, dtype=to, out=(got[0], got[1][:, :64]), dev_err=err)
        assert int(err.item()) == 0
        val = np.full((n, dc + 64), 9.0)
        val[r] = L.values(want)[pg, ln]
        val = val.astype(np.float32)
        for g, w in zip(got, (val[:, :dc], val[:, dc:])):
            assert same(T.host(g)[:, :w.shape[1]], w if to is torch.float32 else T.bf16_round(w))
        assert (got[1][:, 64:] == 9).all()


def test_no_rows(H):
    import torch

    kv = H.KV(k=torch.zeros((1, 1, 64, 576), dtype=torch.bfloat16, device="cuda"), v=None,
              block_table=torch.zeros((1, 1), dtype=torch.int32, device="cuda"),
              seq_len=torch.ones(1, dtype=torch.int32, device="cuda"))
    rs, table = torch.zeros(2, dtype=torch.int32, device="cuda"), T.device(L.rot_table(4, 64))
    z = torch.zeros((0, 576), dtype=torch.bfloat16, device="cuda")
    H.hs2_latent_write(kv, z[:, :512], z[:, 512:], rs, table)
    c, r = H.hs2_latent_read(kv, rs, 0)
    assert c.shape == (0, 512) and r.shape == (0, 64)
    q = torch.zeros((0, 4, 576), dtype=torch.bfloat16, device="cuda")
    o, lse = H.hs2_latent_chunk(q, rs, kv, 1.0, 0)
    assert o.shape == (0, 4, 512) and lse.shape == (0, 4)
