"""Paged-cache operators where calls meet: other streams, pools behind 32-bit offsets, values that
are not finite. Tolerances as in the tests of hs2_fa_chunk."""
import numpy as np
import pytest

import cache_testutil as T
from test_gpu_chunk import H, case, check, run  # noqa: F401

pytestmark = pytest.mark.gpu


def test_results_on_another_stream(H):  # noqa: F811
    """Results and workspaces of a call on a side stream do not lie in memory that work still
    running on the current stream uses."""
    import torch

    lens, counts = [700, 90], [300, 1]
    rng, c, bt, rs, qraw, qval = case(61, "fp4", lens, counts, 8, 1, 128)
    want = T.attend(c, qval, rs, lens, bt, 0.1)
    kv = T.device_cache(H, c, bt, lens)
    q, drs = T.device(qraw), T.device(rs)
    nb = H.hs2_fa_chunk_workspace(len(qraw), 8, kv, 300, 700)
    side = torch.cuda.Stream()
    for _ in range(2):
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        busy = [torch.empty(q.shape, device="cuda") for _ in range(4)]
        busy += [torch.empty(q.shape[:2], device="cuda") for _ in range(4)]
        busy += [torch.empty(nb, dtype=torch.uint8, device="cuda") for _ in range(2)]
        torch.cuda._sleep(20_000_000)  # some 10 ms
        for x in busy:
            x.fill_(255)
        del busy, x
        o, lse = H.hs2_fa_chunk(q, drs, kv, 0.1, 300, max_t=700, stream=side)
        k, v = H.hs2_kv_read(kv, drs, len(qraw), stream=side)
        table, length = H.hs2_pages_fork(*books(H, kv, bt, lens), stream=side)
        torch.cuda.synchronize()
        check((o.double().cpu().numpy(), lse.cpu().numpy()), want, "fp4")
        k2, v2 = H.hs2_kv_read(kv, drs, len(qraw))
        assert torch.equal(k, k2) and torch.equal(v, v2)
        assert length.tolist() == [lens[1], lens[1]] and (table[:, 0] == int(bt[1, 0])).all()
    del rng


def books(H, kv, bt, lens):  # noqa: F811
    """A pool's books for these sequences (the second a full page long at least), and two branches of it."""
    import torch

    n = kv.k.shape[0]
    ref = np.zeros(n, np.int32)
    for b, t in enumerate(lens):
        ref[bt[b, :-(-t // 64)]] = 1
    free = np.full(n, -1, np.int32)
    free[:(ref == 0).sum()] = np.nonzero(ref == 0)[0]
    p = H.Pages(ref=T.device(ref), free_list=T.device(free), n_free=T.device(np.array([(ref == 0).sum()], np.int32)))
    torch.cuda.synchronize()
    return p, [kv], T.device(np.array([1, 1], np.int32))


@pytest.mark.parametrize("dtype,Hkv,num_pages", [("bf16", 8, 33000), ("fp8", 16, 33000), ("fp4", 16, 40000), ("f32", 8, 17000)])
def test_pools_behind_32_bit_offsets(H, dtype, Hkv, num_pages):  # noqa: F811
    """Pages at the end of a pool of more than 2^31 bytes (bf16: channels) give what the same
    pages give in a small pool, on the way in, in attention, in a branch and when they move."""
    import torch

    lens, counts = [200, 65, 130], [130, 1, 66]
    rng, c, bt, rs, qraw, qval = case(62, dtype, lens, counts, 2 * Hkv, Hkv, 128, spare=3)
    P = c["num_pages"]
    small = T.device_cache(H, c, bt, lens)
    off = num_pages - P

    def big_of(t, fill=0):
        if t is None:
            return None
        x = torch.full((num_pages, *t.shape[1:]), fill, dtype=t.dtype, device="cuda")
        x[off:] = t
        return x

    big = H.KV(k=big_of(small.k), v=big_of(small.v), block_table=small.block_table + off, seq_len=small.seq_len,
               k_scale=big_of(small.k_scale, 1), v_scale=big_of(small.v_scale, 1), k_sf=big_of(small.k_sf), v_sf=big_of(small.v_sf))
    assert big.k.nbytes > 2 ** 31
    rows = torch.tensor(rng.standard_normal((len(qraw), Hkv, 128)), dtype=torch.float32, device="cuda")
    q, drs = T.device(qraw), T.device(rs)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    names = ("k", "v", "k_scale", "v_scale", "k_sf", "v_sf")

    def same(a, b):
        for n in names:
            if getattr(a, n) is not None:
                assert torch.equal(getattr(a, n), getattr(b, n)[off:]), n

    for kv in (small, big):
        H.hs2_kv_write(kv, rows, rows.flip(0), drs, dev_err=err)
    same(small, big)
    got = [H.hs2_kv_read(kv, drs, len(qraw), dev_err=err) for kv in (small, big)]
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    for max_n, max_t in ((130, 200), (bt.shape[1] * 64,) * 2):
        o = [H.hs2_fa_chunk(q, drs, kv, 0.1, max_n, max_t=max_t, dev_err=err) for kv in (small, big)]
        assert torch.equal(o[0][0], o[1][0]) and torch.equal(o[0][1], o[1][1])
    # the big pool's sequences move from its end to its front, with their contents
    p = books(H, big, bt + off, lens)[0]
    H.hs2_pages_compact(p, [big], dev_err=err)
    moved = H.hs2_kv_read(big, drs, len(qraw), dev_err=err)
    assert int(big.block_table[0].max()) < P
    assert torch.equal(got[0][0], moved[0]) and torch.equal(got[0][1], moved[1])
    assert int(err.item()) == 0
    del qval


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8", "fp4"])
@pytest.mark.parametrize("n", [2, 60, 300])
def test_a_nan_key_reaches_the_rows_that_see_it(H, dtype, n):  # noqa: F811
    lens, counts = [n + 300, n], [n, n]
    rng, c, bt, rs, qraw, qval = case(63, dtype, lens, counts, 8, 1, 64)
    clean = T.attend(c, qval, rs, lens, bt, 0.125)
    pos = n + 300 - n // 2 - 1  # of sequence 0: the later half of its rows see it
    page, line = bt[0, pos // 64], pos % 64
    if dtype == "f32":
        c["k"][page, 0, line, 5] = np.nan
    elif dtype == "bf16":
        c["k"][page, 0, line, 5] = 0x7FC0
    elif dtype == "fp8":
        c["k"][page, 0, line, 5] = 0x7F
    else:
        c["k_sf"][page, 0, line, 1] = 0x7F
    o, lse, err = run(H, c, bt, lens, rs, qraw, 0.125)
    assert err == 0
    sees = np.zeros(len(qraw), bool)
    sees[pos - 300:n] = True
    assert np.isnan(o[sees]).all() and np.isnan(lse[sees]).all()
    check((o[~sees], lse[~sees]), tuple(x[~sees] for x in clean), dtype)
    del rng


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8", "fp4"])
@pytest.mark.parametrize("max_n,max_t", [(16, 200), (300, 512), (131072, 131072)])
def test_descending_row_starts(H, dtype, max_n, max_t):  # noqa: F811
    """Row starts that fall: flagged on every route, and nothing is written (float32: only rows of
    sequences that the starts give some)."""
    import torch

    lens, counts = [200, 70, 90, 64], [10, 10, 10, 10]
    rng, c, bt, rs, qraw, qval = case(64, dtype, lens, counts, 8, 1, 64, extra=300)
    wide = np.full((4, max(max_t // 64, bt.shape[1])), 10 ** 9, np.int32)
    wide[:, :bt.shape[1]] = bt
    for starts in ([0, 10, 5, 20, 30], [0, 10, -2 ** 31, -5, 10], [0, 2 ** 31 - 1, -2 ** 31, 0, 10]):
        o, lse, err = run(H, c, wide, lens, np.array(starts, np.int32), qraw, 0.1, max_n=max_n, max_t=max_t)
        assert err & H.DEV_BAD_LENGTH
        rows = slice(20 if dtype == "f32" else 0, None)
        assert (o[rows] == 9).all() or dtype == "f32"
        assert np.isfinite(o).all()
    kv = T.device_cache(H, c, wide, lens)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    k, _ = H.hs2_kv_read(kv, T.device(np.array([0, 10, 5, 20, 30], np.int32)), 30, dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) & H.DEV_BAD_LENGTH
    del rng, qval, rs, k
