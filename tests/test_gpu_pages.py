"""The books of a page pool (grow, free, fork, compact) against a plain simulation, and runs of
the paged-cache operators together."""
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


class Books:
    """The plain form: references and the stack of free pages."""

    def __init__(self, num_pages):
        self.ref = np.zeros(num_pages, np.int32)
        self.free = list(range(num_pages - 1, -1, -1))

    def grow(self, table, lens, new):
        old = lens.copy()
        for b in range(len(lens)):
            lens[b] += new[b]
            for j in range(-(-old[b] // 64), -(-lens[b] // 64)):
                table[b, j] = self.free.pop()
                self.ref[table[b, j]] = 1

    def drop(self, table, lens, which):
        gone = set()
        for b in np.nonzero(which)[0]:
            for j in range(-(-lens[b] // 64)):
                p = table[b, j]
                self.ref[p] -= 1
                if self.ref[p] == 0:
                    gone.add(int(p))
        self.free += sorted(gone)

    def fork(self, table, lens, src, pools):
        child = np.full((len(src), table.shape[1]), -1, np.int32)
        length = np.zeros(len(src), np.int32)
        for c, p in enumerate(src):
            if p < 0:
                continue
            length[c] = t = lens[p]
            child[c, :t // 64] = table[p, :t // 64]
            for q in child[c, :t // 64]:
                self.ref[q] += 1
            if t % 64:
                new, old = self.free.pop(), table[p, t // 64]
                child[c, t // 64] = new
                self.ref[new] = 1
                for cache in pools:
                    for name, x in cache.items():
                        if isinstance(x, np.ndarray):
                            if name.endswith("scale"):
                                x[new] = x[old]
                            else:
                                x[new, :, :t % 64] = x[old, :, :t % 64]
        return child, length

    def compact(self, table, lens, pools):
        n, live = len(self.ref), self.ref > 0
        L = int(live.sum())
        to, of = np.nonzero(~live[:L])[0], np.nonzero(live[L:])[0] + L
        place = np.arange(n)
        place[of] = to
        for cache in pools:
            for x in cache.values():
                if isinstance(x, np.ndarray):
                    x[to] = x[of]
        self.ref[to], self.ref[L:] = self.ref[of], 0
        for b, t in enumerate(lens):
            table[b, :-(-t // 64)] = place[table[b, :-(-t // 64)]]
        self.free = list(range(n - 1, L - 1, -1))

    def check(self, pages):
        np.testing.assert_array_equal(pages.ref.cpu().numpy(), self.ref)
        n = int(pages.n_free.item())
        assert n == len(self.free)
        np.testing.assert_array_equal(pages.free_list.cpu().numpy()[:n], self.free)


def dev(x):
    return T.device(np.asarray(x, np.int32))


def test_grow_free_lifecycle(H):
    """Sequences that come, grow by odd amounts and go, for many steps."""
    import torch

    rng = np.random.default_rng(31)
    NP, B, W = 400, 13, 40
    books, pages = Books(NP), H.Pages.make(NP)
    lens, table = np.zeros(B, np.int32), np.full((B, W), -1, np.int32)
    dt, dl = dev(table), dev(lens)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for step in range(25):
        new = rng.choice([0, 1, 5, 63, 64, 65, 300], B).astype(np.int32)
        new = np.where((lens + new) > W * 64, 0, new).astype(np.int32)
        if (-(-(lens + new) // 64) + lens * 0).sum() <= NP:
            books.grow(table, lens, new)
            H.hs2_pages_grow(pages, dt, dl, dev(new), dev_err=err)
        drop = (rng.random(B) < 0.25).astype(np.int32)
        books.drop(table, lens, drop)
        H.hs2_pages_free(pages, dt, dl, dev(drop), dev_err=err)
        for b in np.nonzero(drop)[0]:
            lens[b] = 0
        dl.copy_(dev(lens))
        books.check(pages)
        got = dt.cpu().numpy()
        for b in range(B):
            np.testing.assert_array_equal(got[b, :-(-lens[b] // 64)], table[b, :-(-lens[b] // 64)])
    assert int(err.item()) == 0


@pytest.mark.parametrize("B,NP", [(1, 1), (2500, 3000), (3, 70000)])
def test_grow_and_free_sizes(H, B, NP):
    """More sequences than a block has threads, a pool of one page, long sequences."""
    rng = np.random.default_rng(32)
    W = max(1, NP // B)
    new = rng.integers(0, 64 * W + 1, B).astype(np.int32)
    new[0] = 64 * W
    books, pages = Books(NP), H.Pages.make(NP)
    table, lens = np.full((B, W), -1, np.int32), np.zeros(B, np.int32)
    dt, dl = dev(table), dev(lens)
    books.grow(table, lens, new)
    H.hs2_pages_grow(pages, dt, dl, dev(new))
    books.check(pages)
    np.testing.assert_array_equal(dt.cpu().numpy(), table)
    np.testing.assert_array_equal(dl.cpu().numpy(), lens)
    drop = np.ones(B, np.int32)
    drop[B // 2 + 1:] = 0
    books.drop(table, lens, drop)
    H.hs2_pages_free(pages, dt, dl, dev(drop))
    books.check(pages)


def test_grow_refuses_what_does_not_fit(H):
    import torch

    pages = H.Pages.make(3)
    dt, dl = dev(np.full((3, 4), -1)), dev([0, 10, 0])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    H.hs2_pages_grow(pages, dt, dl, dev([64, 0, 129]), dev_err=err)  # four pages of three
    assert int(err.item()) == H.DEV_BAD_PAGE
    assert (dt == -1).all() and dl.tolist() == [0, 10, 0] and int(pages.n_free) == 3 and (pages.ref == 0).all()
    err.zero_()
    H.hs2_pages_grow(pages, dt, dl, dev([257, -1, 100]), dev_err=err)  # beyond the table; negative; fine
    assert int(err.item()) == H.DEV_BAD_LENGTH
    assert dl.tolist() == [0, 10, 100] and dt[2].tolist() == [0, 1, -1, -1] and int(pages.n_free) == 1


def test_free_flags_pages_without_references(H):
    """A page freed twice, an entry out of range and a bad length: flagged, nothing pushed twice."""
    import torch

    pages = H.Pages.make(4)
    dt, dl = dev(np.full((3, 2), -1)), dev([0, 0, 0])
    H.hs2_pages_grow(pages, dt, dl, dev([128, 0, 0]))
    dt[1, 0], dt[1, 1], dl[1], dl[2] = 0, 9, 128, 129  # sequence 1 claims page 0 too
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    H.hs2_pages_free(pages, dt, dl, dev([1, 1, 1]), dev_err=err)
    assert int(err.item()) == H.DEV_BAD_PAGE | H.DEV_BAD_LENGTH
    assert pages.ref.tolist() == [0, 0, 0, 0] and int(pages.n_free) == 4
    assert sorted(pages.free_list.tolist()) == [0, 1, 2, 3]


@pytest.mark.parametrize("dtypes", [("bf16",), ("fp4", "f32"), ("fp8", "bf16", "fp4")])
def test_fork_shares_and_copies(H, dtypes):
    import torch

    rng = np.random.default_rng(33)
    NP, lens = 60, np.array([64, 65, 0, 200, 1, 128, 383], np.int32)
    books, pages = Books(NP), H.Pages.make(NP)
    pools = [T.make_cache(rng, t, NP, h, d, key_only=i == 2) for i, (t, h, d) in
             enumerate(zip(dtypes, (2, 1, 3), (64, 128, 64)))]
    table, zero = np.full((len(lens), 8), -1, np.int32), np.zeros(len(lens), np.int32)
    dt, dl = dev(table), dev(zero)
    books.grow(table, zero, lens)
    H.hs2_pages_grow(pages, dt, dl, dev(lens))
    kvs = []
    for c in pools:
        kv = T.device_cache(H, c, table, lens)
        kv.block_table, kv.seq_len = dt, dl
        kvs.append(kv)
    src = np.array([3, 3, -1, 1, 6, 0, 2, 4, 3, 5, 6], np.int32)
    child, length = books.fork(table, lens, src, pools)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    gt, gl = H.hs2_pages_fork(pages, kvs, dev(src), dev_err=err)
    assert int(err.item()) == 0
    np.testing.assert_array_equal(gt.cpu().numpy(), child)
    np.testing.assert_array_equal(gl.cpu().numpy(), length)
    books.check(pages)
    for kv, c in zip(kvs, pools):
        got = T.cache_arrays(kv, c)
        for name in got:
            np.testing.assert_array_equal(got[name], c[name], err_msg=name)
    # the sources end, then the branches: every page comes back
    books.drop(table, lens, np.ones(len(lens)))
    H.hs2_pages_free(pages, dt, dl, dev(np.ones(len(lens))), dev_err=err)
    books.check(pages)
    books.drop(child, length, np.ones(len(src)))
    H.hs2_pages_free(pages, gt, gl, dev(np.ones(len(src))), dev_err=err)
    books.check(pages)
    assert int(err.item()) == 0 and int(pages.n_free) == NP


def test_fork_refusals(H):
    import torch

    rng = np.random.default_rng(34)
    c = T.make_cache(rng, "bf16", 5, 1, 64)
    pages = H.Pages.make(5)
    dt, dl = dev(np.full((3, 3), -1)), dev([0, 0, 0])
    H.hs2_pages_grow(pages, dt, dl, dev([100, 64, 0]))
    kv = T.device_cache(H, c, np.zeros((3, 3)), [0, 0, 0])
    kv.block_table, kv.seq_len = dt, dl
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    t, n = H.hs2_pages_fork(pages, [kv], dev([0, 0, 0]), dev_err=err)  # three pages of two
    assert int(err.item()) == H.DEV_BAD_PAGE and (t == -1).all() and (n == 0).all() and int(pages.n_free) == 2
    err.zero_()
    dl[2] = 193  # longer than the table
    t, n = H.hs2_pages_fork(pages, [kv], dev([3, -2, 2, 1]), dev_err=err)
    assert int(err.item()) == H.DEV_BAD_INDEX | H.DEV_BAD_LENGTH and n.tolist() == [0, 0, 0, 64]
    assert pages.ref.tolist()[int(t[3, 0])] == 2
    err.zero_()
    dt[1, 0] = 7
    t, n = H.hs2_pages_fork(pages, [kv], dev([1]), dev_err=err)
    assert int(err.item()) == H.DEV_BAD_PAGE and t[0, 0] == -1
    with pytest.raises(H.HS2Error):  # another pool size
        H.hs2_pages_fork(H.Pages.make(6), [kv], dev([1]))


@pytest.mark.parametrize("NP,B,seed", [(50, 6, 1), (1, 1, 2), (3000, 40, 3), (20011, 90, 4)])
def test_compact(H, NP, B, seed):
    import torch

    rng = np.random.default_rng(seed)
    big = NP > 1000
    pools = [T.make_cache(rng, "fp4", NP, 1, 64)] + ([] if big else [T.make_cache(rng, "bf16", NP, 2, 128)])
    W = max(1, NP // B)
    lens = rng.integers(0, 64 * W + 1, B).astype(np.int32)
    table = T.make_table(rng, lens, NP, W)
    books, pages = Books(NP), H.Pages.make(NP)
    keep = rng.random(B) < 0.5
    if B == 1:
        keep[:] = True
    lens, table = lens[keep], table[keep]
    if len(lens) > 1 and lens[0] >= 64 and lens[1] >= 64:
        table[1, 0] = table[0, 0]  # a shared page
    for b, t in enumerate(lens):
        for p in table[b, :-(-t // 64)]:
            books.ref[p] += 1
    books.free = [int(p) for p in rng.permutation(np.nonzero(books.ref == 0)[0])]
    pages.ref.copy_(dev(books.ref))
    if books.free:
        pages.free_list[:len(books.free)] = dev(books.free)
    pages.n_free.fill_(len(books.free))
    kvs = []
    dt, dl = dev(table), dev(lens)
    for c in pools:
        kv = T.device_cache(H, c, table, lens)
        kv.block_table, kv.seq_len = dt, dl
        kvs.append(kv)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    books.compact(table, lens, pools)
    H.hs2_pages_compact(pages, kvs, dev_err=err)
    assert int(err.item()) == 0
    books.check(pages)
    np.testing.assert_array_equal(dt.cpu().numpy(), table)
    for kv, c in zip(kvs, pools):
        got = T.cache_arrays(kv, c)
        for name in got:
            np.testing.assert_array_equal(got[name], c[name], err_msg=name)
    H.hs2_pages_compact(pages, kvs, dev_err=err)  # a compact pool stays as it is
    books.check(pages)
    np.testing.assert_array_equal(dt.cpu().numpy(), table)
    assert int(err.item()) == 0


def test_compact_leaves_bad_entries(H):
    import torch

    rng = np.random.default_rng(36)
    c = T.make_cache(rng, "fp8", 6, 1, 64)
    pages = H.Pages.make(6)
    pages.ref.copy_(dev([0, 1, 0, 0, 1, 0]))
    dt, dl = dev([[4, 1, -5], [5, 4, 4]]), dev([192, 500])
    kv = T.device_cache(H, c, np.zeros((2, 3)), [0, 0])
    kv.block_table, kv.seq_len = dt, dl
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    H.hs2_pages_compact(pages, [kv], dev_err=err)
    assert int(err.item()) == H.DEV_BAD_PAGE | H.DEV_BAD_LENGTH
    assert dt.tolist() == [[0, 1, -5], [5, 4, 4]] and pages.ref.tolist() == [1, 1, 0, 0, 0, 0]
    assert int(pages.n_free) == 4 and pages.free_list.tolist() == [5, 4, 3, 2, -1, -1]


@pytest.mark.parametrize("dtype", ["fp4", "fp8", "bf16"])
@pytest.mark.parametrize("captured", [False, True])
def test_serving_run(H, dtype, captured):
    """Prompts admitted, written and attended; branches forked, grown by a draft token each and
    verified; the pool compacted; the branches attend again and end. Captured: each step's graph
    is replayed on other inputs than it was captured with. Attention against the 64-bit form on the
    rows as they were written."""
    import torch

    rng = np.random.default_rng(41)
    NP, Hq, Hkv, d, W = 64, 8, 2, 64, 12
    counts = [70, 1, 64, 130]
    c = T.make_cache(rng, dtype, NP, Hkv, d, scale=1.0)
    pages = H.Pages.make(NP)
    dt, dl = dev(np.full((4, W), -1)), dev(np.zeros(4))
    kv = T.device_cache(H, c, np.zeros((4, W)), np.zeros(4))
    kv.block_table, kv.seq_len = dt, dl
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    n, rs = sum(counts), dev(T.starts(counts))
    rows = [torch.zeros((n, Hkv, d), device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    q = torch.zeros((n, Hq, d), device="cuda", dtype=torch.bfloat16)
    src = dev([3, 3, 0, -1, 1])
    ct, cl = torch.empty((5, W), device="cuda", dtype=torch.int32), torch.empty(5, device="cuda", dtype=torch.int32)
    ckv = H.KV(k=kv.k, v=kv.v, block_table=ct, seq_len=cl, k_scale=kv.k_scale, v_scale=kv.v_scale, k_sf=kv.k_sf,
               v_sf=kv.v_sf)
    drs = dev(T.starts([1, 1, 1, 0, 1]))
    drows = [torch.zeros((4, Hkv, d), device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    dq = torch.zeros((4, Hq, d), device="cuda", dtype=torch.bfloat16)
    one = dev([1, 1, 1, 0, 1])
    out = [torch.empty((m, Hq, d), device="cuda") for m in (n, 4, 4)]
    lse = [torch.empty((m, Hq), device="cuda") for m in (n, 4, 4)]
    every, none4 = dev(np.ones(5)), dev(counts)
    stream = torch.cuda.Stream()

    ws = [torch.empty(H.hs2_fa_chunk_workspace(m, Hq, k, 130, W * 64), device="cuda", dtype=torch.uint8)
          for m, k in ((n, kv), (4, ckv))]
    cws = torch.empty(H.hs2_pages_compact_workspace(pages), device="cuda", dtype=torch.uint8)
    both = torch.empty((9, W), device="cuda", dtype=torch.int32)  # all sequences of the pool, for compaction
    blen = torch.empty(9, device="cuda", dtype=torch.int32)
    bkv = H.KV(k=kv.k, v=kv.v, block_table=both, seq_len=blen, k_scale=kv.k_scale, v_scale=kv.v_scale, k_sf=kv.k_sf,
               v_sf=kv.v_sf)

    def step():
        H.hs2_pages_grow(pages, dt, dl, none4, dev_err=err)
        H.hs2_kv_write(kv, rows[0], rows[1], rs, dev_err=err)
        H.hs2_fa_chunk(q, rs, kv, 0.125, 130, out=(out[0], lse[0]), workspace=ws[0], dev_err=err)
        H.hs2_pages_fork(pages, [kv], src, out=(ct, cl), dev_err=err)
        H.hs2_pages_grow(pages, ct, cl, one, dev_err=err)
        H.hs2_kv_write(ckv, drows[0], drows[1], drs, dev_err=err)
        H.hs2_fa_chunk(dq, drs, ckv, 0.125, 1, out=(out[1], lse[1]), workspace=ws[1], dev_err=err)
        both[:4].copy_(dt)
        both[4:].copy_(ct)
        blen[:4].copy_(dl)
        blen[4:].copy_(cl)
        H.hs2_pages_compact(pages, [bkv], workspace=cws, dev_err=err)
        dt.copy_(both[:4])
        ct.copy_(both[4:])
        H.hs2_fa_chunk(dq, drs, ckv, 0.125, 1, out=(out[2], lse[2]), workspace=ws[1], dev_err=err)
        H.hs2_pages_free(pages, dt, dl, every[:4], dev_err=err)
        H.hs2_pages_free(pages, ct, cl, every, dev_err=err)
        dl.zero_()

    graph = None
    if captured:
        with torch.cuda.stream(stream):
            step()
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
    for trial in range(2):
        for t in (*rows, q, *drows, dq):
            t.copy_(torch.from_numpy(rng.standard_normal(t.shape).astype(np.float32)))
        torch.cuda.synchronize()
        if graph is not None:
            graph.replay()
        else:
            step()
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        assert int(pages.n_free) == NP and (pages.ref == 0).all()
        # the plain form: one sequence per entry, rows written in order; slab scales differ by page, so the
        # values are read back from where the rows of the first attention were written
        val = {}
        for side, x in zip(("k", "v"), rows):
            val[side] = x.float().cpu().numpy().astype(np.float64)
        for side, x in zip(("k", "v"), drows):
            val["d" + side] = x.float().cpu().numpy().astype(np.float64)
        if dtype == "bf16":
            plain = {"dtype": "f32", "Hkv": Hkv, "d": d, "num_pages": 64}
            kids = [(3, 0), (3, 1), (0, 2), (1, 3)]
            bt0 = T.make_table(np.random.default_rng(1), counts + [counts[p] + 1 for p, _ in kids], 64, W)
            for side in ("k", "v"):
                pool = np.zeros((64, Hkv, 64, d), np.float32)
                at = T.starts(counts)
                for b, t in enumerate(counts):
                    for i in range(t):
                        pool[bt0[b, i // 64], :, i % 64] = val[side][at[b] + i]
                plain[side] = pool
            qv = q.float().cpu().numpy().astype(np.float64)
            ro, rlse, mag = T.attend(plain, qv, T.starts(counts), counts, bt0, 0.125)
            assert (np.abs(out[0].cpu().numpy() - ro) <= (2.0 ** -8 + 1e-3) * mag + 1e-6).all()
            for i, (p, row) in enumerate(kids):
                t, b = counts[p] + 1, 4 + i
                for side in ("k", "v"):
                    at = T.starts(counts)
                    for j in range(t):
                        x = val[side][at[p] + j] if j < t - 1 else val["d" + side][row]
                        plain[side][bt0[b, j // 64], :, j % 64] = x
                one_q = dq[row:row + 1].float().cpu().numpy().astype(np.float64)
                ro, rlse, mag = T.attend(plain, one_q, T.starts([1]), [t], bt0[b:b + 1], 0.125)
                for o in out[1:]:
                    assert (np.abs(o[row].cpu().numpy() - ro[0]) <= (2.0 ** -8 + 1e-3) * mag[0] + 1e-6).all()
        # moved pages are read like the ones before the move
        assert torch.equal(out[1], out[2]) and torch.equal(lse[1], lse[2])
