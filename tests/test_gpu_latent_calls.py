"""Calls of the latent operators and of the rotated rows that the documentation allows: outputs on 16
bytes, without lse, no rows, rows in graphs and on side streams, page books of every latent cache."""
import numpy as np
import pytest

import cache_testutil as T
import latent_testutil as L
from test_gpu_latent import (H, SCALE, check, expanded_case, latent_case, latent_kv, run, run_expanded,  # noqa: F401
                             want_expanded)

pytestmark = pytest.mark.gpu

EXPANDED = [(4, [300, 5], [300, 700]), (16, [40], [3000]), (2, [40] * 40, [1200] * 40)]
ABSORBED = [(16, [700, 300], [2, 1]), (128, [5000, 3], [1, 1]), (64, [1300, 900], [90, 1])]


def off_32(shape, dtype):
    """A contiguous tensor of 9s that starts on 16 bytes but not on 32, and what surrounds it."""
    import torch

    n, step = int(np.prod(shape)), 16 // torch.empty(0, dtype=dtype).element_size()
    whole = torch.full((n + 2 * step,), 9.0, dtype=dtype, device="cuda")
    x = whole[step:step + n].view(shape)
    assert x.data_ptr() % 32 == 16
    return x, (whole[:step], whole[step + n:])


@pytest.mark.parametrize("o_type", ["f32", "bf16"])
@pytest.mark.parametrize("Hq,counts,keys", EXPANDED)
def test_expanded_outputs_on_16_bytes(H, o_type, Hq, counts, keys):  # noqa: F811
    import torch

    o_dtype = torch.float32 if o_type == "f32" else torch.bfloat16
    rng, rs, ks, q, kv, r = expanded_case(81, "bf16", counts, keys, Hq)
    d = T.device(kv)
    args = (T.device(q), d[..., :128], T.device(r), d[..., 128:], T.device(rs), T.device(ks), SCALE, max(counts), max(keys))
    o, around = off_32((len(q), Hq, 128), o_dtype)
    lse = torch.zeros((len(q), Hq), device="cuda")
    H.hs2_latent_prefill(*args, o_dtype=o_dtype, out=(o, lse))
    check((o.double().cpu().numpy(), lse.cpu().numpy()), want_expanded(rs, ks, q, kv, r), "bf16", 192, o_bf16=o_type == "bf16")
    assert all((x == 9).all() for x in around)
    plain = H.hs2_latent_prefill(*args, o_dtype=o_dtype)
    no_lse = torch.zeros_like(plain[0])
    assert H.hs2_latent_prefill(*args, o_dtype=o_dtype, out=(no_lse, None))[1] is None
    assert torch.equal(plain[0], o) and torch.equal(plain[0], no_lse) and torch.equal(plain[1], lse)


@pytest.mark.parametrize("dtype,o_type", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
@pytest.mark.parametrize("Hq,lens,counts", ABSORBED)
def test_absorbed_outputs_on_16_bytes(H, dtype, o_type, Hq, lens, counts):  # noqa: F811
    import torch

    o_dtype = torch.float32 if o_type == "f32" else torch.bfloat16
    rng, pool, bt, rs, q = latent_case(82, dtype, lens, counts, Hq, 256)
    args = (T.device(q), T.device(rs), latent_kv(H, pool, bt, lens), SCALE, max(counts))
    o, around = off_32((len(q), Hq, 256), o_dtype)
    lse = torch.zeros((len(q), Hq), device="cuda")
    H.hs2_latent_chunk(*args, max_t=max(lens), o_dtype=o_dtype, out=(o, lse))
    want = L.absorbed(L.values(pool), L.values(q), rs, lens, bt, SCALE)
    check((o.double().cpu().numpy(), lse.cpu().numpy()), want, dtype, 320, o_bf16=o_type == "bf16")
    assert all((x == 9).all() for x in around)
    plain = H.hs2_latent_chunk(*args, max_t=max(lens), o_dtype=o_dtype)
    no_lse = torch.zeros_like(plain[0])
    assert H.hs2_latent_chunk(*args, max_t=max(lens), o_dtype=o_dtype, out=(no_lse, None))[1] is None
    assert torch.equal(plain[0], o) and torch.equal(plain[0], no_lse) and torch.equal(plain[1], lse)


def test_f32_without_lse(H):  # noqa: F811
    import torch

    rng, rs, ks, q, kv, r = expanded_case(83, "f32", [70, 3], [200, 131], 3)
    d = T.device(kv)
    args = (T.device(q), d[..., :128], T.device(r), d[..., 128:], T.device(rs), T.device(ks), SCALE, 70, 200)
    plain = H.hs2_latent_prefill(*args)
    o = torch.zeros_like(plain[0])
    H.hs2_latent_prefill(*args, out=(o, None))
    assert torch.equal(o, plain[0])


@pytest.mark.parametrize("counts,keys,Hq", [([500, 5], [700, 300], 4), ([40], [3000], 16)])
def test_expanded_on_streams(H, counts, keys, Hq):  # noqa: F811
    """Two calls at once, a workspace each, bit for bit as alone."""
    import torch

    rng, rs, ks, q, kv, r = expanded_case(84, "bf16", counts, keys, Hq)
    d, dq, dr, drs, dks = T.device(kv), T.device(q), T.device(r), T.device(rs), T.device(ks)
    call = lambda x, **kw: H.hs2_latent_prefill(x, d[..., :128], dr, d[..., 128:], drs, dks, SCALE, max(counts), max(keys), **kw)  # noqa: E731
    other = (dq * 0.5).contiguous()
    want = call(dq), call(other)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[call(x, stream=s) for x, s in zip((dq, other), streams)] for _ in range(5)]
    torch.cuda.synchronize()
    for pair in got:
        for a, b in zip(pair, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ---------------------------------------------------------------------------- rows
def row_calls(H, rng, dtype, n):  # noqa: F811
    """(name, inputs that a new step overwrites, call, outputs) of either kind of rows; queries in place too."""
    import torch

    lens, counts = [n + 70, 64], [n, 64]
    rs, pages = T.starts(counts), sum(-(-t // 64) for t in (n + 70, 64))
    rows = int(rs[-1])
    bt = T.make_table(rng, lens, pages)
    table, drs, dlen = T.device(L.rot_table(max(lens), 64)), T.device(rs), T.device(np.array(lens, np.int32))
    c = T.make_cache(rng, dtype, pages, 2, 64)
    kv = T.device_cache(H, c, bt, lens)
    x = torch.randn((rows, 2 + 2 + 5, 64), device="cuda").to(torch.bfloat16)
    q_out = torch.zeros((rows, 5, 64), device="cuda", dtype=torch.bfloat16)
    pools = [t for t in (kv.k, kv.v, kv.k_sf, kv.v_sf) if t is not None]
    yield x, lambda **kw: H.hs2_kv_write_rot(kv, x[:, :2], x[:, 2:4], drs, table, q=x[:, 4:], q_out=q_out, **kw), pools + [q_out]
    lat = H.KV(k=torch.zeros((pages, 1, 64, 576), device="cuda", dtype=torch.bfloat16), v=None, block_table=T.device(bt),
               seq_len=dlen)
    y = torch.randn((rows, 576 + 9 * 64), device="cuda").to(torch.bfloat16)
    to = torch.zeros((rows, 9, 576), device="cuda", dtype=torch.bfloat16)
    back = torch.zeros((rows, 512), device="cuda", dtype=torch.bfloat16), torch.zeros((rows, 64), device="cuda", dtype=torch.bfloat16)

    def both(**kw):
        H.hs2_latent_write(lat, y[:, :512], y[:, 512:576], drs, table, q=y[:, 576:].unflatten(1, (9, 64)), q_out=to[..., 512:], **kw)
        H.hs2_latent_read(lat, drs, rows, out=back, **kw)

    yield y, both, [lat.k, to, *back]


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("n", [3, 7300])
def test_rows_in_graphs_and_on_streams(H, dtype, n):  # noqa: F811
    """Captured and replayed with new rows in place, and on a side stream, bit for bit as eager."""
    import torch

    for x, call, outs in row_calls(H, np.random.default_rng(85), dtype, n):
        start = [t.clone() for t in outs]
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        old = [t.clone() for t in outs]
        x.copy_(torch.randn_like(x.float()).to(x.dtype))
        call()
        torch.cuda.synchronize()
        want = [t.clone() for t in outs]
        assert not any(torch.equal(a, b) for a, b in zip(old, want))
        side = torch.cuda.Stream()
        for again in (g.replay, lambda: call(stream=side)):
            for t, was in zip(outs, start):
                t.copy_(was)
            torch.cuda.synchronize()
            again()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_no_rows_with_queries(H):  # noqa: F811
    """Empty arrays, queries among them, are no error."""
    import torch

    bf = dict(dtype=torch.bfloat16, device="cuda")
    ints = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    rs, table = ints(2), T.device(L.rot_table(4, 64))
    lat = H.KV(k=torch.zeros((1, 1, 64, 576), **bf), v=None, block_table=ints(1, 1), seq_len=ints(1) + 1)
    z, q, to = torch.zeros((0, 576), **bf), torch.zeros((0, 16, 192), **bf), torch.zeros((0, 16, 576), **bf)
    got = H.hs2_latent_write(lat, z[:, :512], z[:, 512:], rs, table, q=q[..., 128:], q_out=to[..., 512:])
    assert got.shape == (0, 16, 64)
    assert H.hs2_latent_write(lat, z[:, :512], z[:, 512:], rs, table, q=q[..., 128:]).shape == (0, 16, 64)
    kv = H.KV(k=torch.zeros((1, 2, 64, 64), **bf), v=torch.zeros((1, 2, 64, 64), **bf), block_table=ints(1, 1), seq_len=ints(1) + 1)
    rows, q = torch.zeros((0, 2, 64), **bf), torch.zeros((0, 4, 64), **bf)
    assert H.hs2_kv_write_rot(kv, rows, rows, rs, table, q=q).shape == (0, 4, 64)
    assert H.hs2_kv_write_rot(kv, rows, rows, rs, table, q=q, q_out=q) is q
    o, lse = H.hs2_latent_prefill(torch.zeros((0, 4, 192), **bf), torch.zeros((0, 4, 128), **bf), torch.zeros((0, 64), **bf),
                                  torch.zeros((0, 4, 128), **bf), rs, rs, 1.0, 0, 0)
    assert o.shape == (0, 4, 128) and lse.shape == (0, 4)
    torch.cuda.synchronize()
    assert (lat.k == 0).all() and (kv.k == 0).all()


# ---------------------------------------------------------------------------- pages
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dc", [512, 256])
def test_books_of_latent_caches(H, dtype, dc):  # noqa: F811
    """Fork, free and compact of every latent cache, beside a K/V cache on the same table."""
    import torch

    rng = np.random.default_rng(86)
    lens, num_pages = [130, 64, 300, 1], 24
    books = H.Pages.make(num_pages)
    bt, sl = torch.full((4, 5), -1, dtype=torch.int32, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    H.hs2_pages_grow(books, bt, sl, T.device(np.array(lens, np.int32)), dev_err=err)
    pool = T.device(L.raw(rng.standard_normal((num_pages, 1, 64, dc + 64)), dtype))
    c = T.make_cache(rng, "bf16", num_pages, 2, 64)
    lat = H.KV(k=pool, v=None, block_table=bt, seq_len=sl)
    kv = H.KV(k=T.device(c["k"]), v=T.device(c["v"]), block_table=bt, seq_len=sl)
    to = torch.float32 if dtype == "f32" else torch.bfloat16
    ks = T.device(T.starts(lens))

    def rows(of, other, starts, n):
        return (*H.hs2_latent_read(of, starts, n, dtype=to, dev_err=err), *H.hs2_kv_read(other, starts, n, dtype=torch.bfloat16, dev_err=err))

    before = rows(lat, kv, ks, sum(lens))
    src = np.array([2, 0, 2], np.int32)
    child_bt, child_len = H.hs2_pages_fork(books, [lat, kv], T.device(src), dev_err=err)
    child = [H.KV(k=x.k, v=x.v, block_table=child_bt, seq_len=child_len) for x in (lat, kv)]
    cl = [lens[s] for s in src]
    got = rows(*child, T.device(T.starts(cl)), sum(cl))
    at = T.starts(lens)
    pick = np.concatenate([np.arange(at[s], at[s + 1]) for s in src])
    for a, b in zip(got, before):
        assert torch.equal(a, b[torch.from_numpy(pick).cuda()])
    H.hs2_pages_free(books, bt, sl, T.device(np.array([1, 1, 0, 1], np.int32)), dev_err=err)
    # what is left of both tables, as one
    left_bt, left_len = torch.cat((bt[2:3], child_bt)).contiguous(), torch.cat((sl[2:3], child_len)).contiguous()
    left = [H.KV(k=x.k, v=x.v, block_table=left_bt, seq_len=left_len) for x in (lat, kv)]
    H.hs2_pages_compact(books, left, dev_err=err)
    ll = [lens[2]] + cl
    got = rows(*left, T.device(T.starts(ll)), sum(ll))
    pick = np.concatenate([np.arange(at[s], at[s + 1]) for s in [2, *src]])
    for a, b in zip(got, before):
        assert torch.equal(a, b[torch.from_numpy(pick).cuda()])
    used = int((books.ref > 0).sum())
    assert int((books.ref[:used] > 0).sum()) == used and int(err.item()) == 0
