"""Latent attention, absorbed and expanded, against the 64-bit forms.

Tolerances, from the roundings on the way (u = half a step: bf16 2^-8, fp32 2^-24):
 lse  a logit is a sum of d exact products in fp32, each addition off by at most 2^-23 of the sum so
      far: d * 2^-23 * scale * sum |q k|. For N(0, 1) inputs and scale 192^-1/2 sum |q k| stays below
      0.87 d (its mean is 0.64 d): 576 * 2^-23 * 36 = 2.5e-3, 192 * 2^-23 * 12 = 2.8e-4; exp2, log2
      and the sums add a few 2^-22.
 o    the weights enter P.V rounded to bf16 (float32: not): off by u * sum p |v| / Z, plus twice the
      logits' errors, plus u |o| where o is bfloat16."""
import numpy as np
import pytest

import cache_testutil as T
import latent_testutil as L

pytestmark = pytest.mark.gpu
SCALE = 192 ** -0.5


def lse_tol(d):
    return d * 2.0 ** -23 * SCALE * 0.87 * d + 1e-5


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


def check(got, want, dtype, d, o_bf16=False, rows=slice(None)):
    (o, lse), (ro, rlse, mag) = got, want
    tol = ((0 if dtype == "f32" else 2.0 ** -8) + 2 * lse_tol(d)) * mag + (2.0 ** -8 * np.abs(ro) if o_bf16 else 0) + 1e-6
    worst = (np.abs(o - ro) - tol)[rows]
    assert worst.size == 0 or worst.max() <= 0, (worst.max(), np.unravel_index(worst.argmax(), worst.shape))
    if lse is not None:
        fin = np.isfinite(rlse[rows])
        assert (np.isfinite(lse[rows]) == fin).all()
        assert np.abs(lse[rows][fin] - rlse[rows][fin]).max(initial=0) <= lse_tol(d)


# ---------------------------------------------------------------------------- absorbed
def latent_case(seed, dtype, lens, counts, Hq, dc, first=0, extra=0, spare=2, width=None):
    rng = np.random.default_rng(seed)
    pages = sum(-(-max(t, 0) // 64) for t in lens) + spare
    pool = L.raw(rng.standard_normal((pages, 64, dc + 64)), dtype)
    bt = T.make_table(rng, lens, pages, width)
    rs = T.starts(counts, first)
    q = L.raw(rng.standard_normal((int(rs[-1]) + extra, Hq, dc + 64)), dtype)
    return rng, pool, bt, rs, q


def poison(pool, bt, lens):
    """NaN in every row that no sequence sees (behind its end, and in pages of nobody)."""
    seen = np.zeros(pool.shape[:2], bool)
    for b, t in enumerate(lens):
        s = np.arange(t)
        page = bt[b, s // 64]
        ok = (page >= 0) & (page < len(pool))
        seen[page[ok], s[ok] % 64] = True
    pool[~seen] = 0x7FC0 if pool.dtype == np.uint16 else np.nan
    return pool


def latent_kv(H, pool, bt, lens):
    return H.KV(k=T.device(pool[:, None]), v=None, block_table=T.device(np.asarray(bt, np.int32)),
                seq_len=T.device(np.asarray(lens, np.int32)))


def run(H, pool, bt, lens, rs, q, scale=SCALE, o_dtype=None, max_n=None, max_t=None, lse=True, **kw):
    import torch

    o_dtype = o_dtype or torch.float32
    n, Hq, d = q.shape
    out = (torch.full((n, Hq, d - 64), 9.0, device="cuda", dtype=o_dtype),
           torch.full((n, Hq), 9.0, device="cuda") if lse else None)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    H.hs2_latent_chunk(T.device(q), T.device(rs), latent_kv(H, pool, bt, lens), scale,
                       max_n if max_n is not None else int(np.diff(rs).max()),
                       max_t=max_t if max_t is not None else int(max(lens)), o_dtype=o_dtype, out=out, dev_err=err, **kw)
    torch.cuda.synchronize()
    return out[0].double().cpu().numpy(), out[1].cpu().numpy() if lse else None, int(err.item())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Hq,dc", [(1, 512), (2, 256), (8, 512), (16, 512), (32, 256), (64, 512), (128, 512), (128, 256)])
def test_ragged_heads(H, dtype, Hq, dc):
    lens, counts = [1, 130, 64, 300, 65, 7, 0, 128, 129], [1, 1, 64, 37, 0, 7, 0, 2, 1]
    rng, pool, bt, rs, q = latent_case(31, dtype, lens, counts, Hq, dc, first=1, extra=2)
    pool = poison(pool, bt, lens)
    want = L.absorbed(L.values(pool), L.values(q), rs, lens, bt, SCALE)
    o, lse, err = run(H, pool, bt, lens, rs, q)
    assert err == 0
    check((o, lse), want, dtype, dc + 64, rows=slice(rs[0], rs[-1]))
    for outside in (slice(0, rs[0]), slice(rs[-1], None)):  # rows of nobody stay as they were
        assert (o[outside] == 9).all() and (lse[outside] == 9).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Hq", [16, 64, 128])
def test_single_tokens(H, dtype, Hq):
    """One token a sequence, lengths about the borders of pages and tiles."""
    import torch

    lens = [1, 2, 63, 64, 65, 127, 128, 129, 191, 192, 193, 255, 256, 257, 511, 1025]
    rng, pool, bt, rs, q = latent_case(32, dtype, lens, [1] * len(lens), Hq, 512)
    pool = poison(pool, bt, lens)
    want = L.absorbed(L.values(pool), L.values(q), rs, lens, bt, SCALE)
    o, lse, err = run(H, pool, bt, lens, rs, q, o_dtype=torch.bfloat16)
    assert err == 0
    check((o, lse), want, dtype, 576, o_bf16=True)


@pytest.mark.parametrize("Hq,lens,counts", [(16, [9000], [1]), (16, [5000, 77], [4, 3]), (128, [7001, 400], [1, 1]),
                                            (32, [3000] * 5, [1, 2, 3, 4, 5]), (128, [2500], [9]), (1, [20000, 3], [1, 3]),
                                            (64, [640] * 40, [1] * 40), (8, [1500, 1500], [200, 130]),
                                            (64, [1300, 900], [90, 1])])
def test_long_and_shared_out(H, Hq, lens, counts):
    """Sequences that several blocks share, chunks of several tiles' rows, more sequences than blocks' worth."""
    rng, pool, bt, rs, q = latent_case(33, "bf16", lens, counts, Hq, 512)
    want = L.absorbed(L.values(pool), L.values(q), rs, lens, bt, SCALE)
    o, lse, err = run(H, pool, bt, lens, rs, q)
    assert err == 0
    check((o, lse), want, "bf16", 576)


@pytest.mark.parametrize("Hq", [16, 64, 128])
@pytest.mark.parametrize("order", ["rising", "falling", "spikes"])
def test_logits_that_grow(H, Hq, order):
    """The running reference moves: logits rise along the keys by hundreds, fall, or leap at single keys."""
    lens, counts = [700, 300], [2, 1]
    rng, pool, bt, rs, q = latent_case(34, "bf16", lens, counts, Hq, 512)
    val = L.values(pool).astype(np.float32)
    lead = np.zeros((576,), np.float32)
    lead[:8] = 1.0
    qv = L.values(q).astype(np.float32)
    qv[..., :8] = 4.0
    for b, t in enumerate(lens):
        s = np.arange(t)
        amount = {"rising": s / t * 300, "falling": (t - s) / t * 300, "spikes": (s % 130 == 129) * (s + 100.0)}[order]
        val[bt[b, s // 64], s % 64, :8] = amount[:, None]  # 32 * amount / sqrt(192) more in the logit
    pool, q = L.raw(val, "bf16"), L.raw(qv, "bf16")
    want = L.absorbed(L.values(pool), L.values(q), rs, lens, bt, SCALE)
    o, lse, err = run(H, pool, bt, lens, rs, q)
    assert err == 0
    # the logits reach 32 * 800 / sqrt(192) = 1850: 576 additions of 2^-23 of that each, at most
    slack = 576 * 2.0 ** -23 * 1850
    ro, rlse, mag = want
    assert (np.abs(lse - rlse) <= slack + 1e-3).all()
    assert (np.abs(o - ro) <= (2.0 ** -8 + 2 * slack) * mag + 1e-6).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Hq", [16, 128])
def test_bad_pages(H, dtype, Hq):
    lens, counts = [300, 64, 129, 500], [3, 1, 2, 1]
    rng, pool, bt, rs, q = latent_case(35, dtype, lens, counts, Hq, 256)
    bt[0, 1] = len(pool)  # the middle of a sequence
    bt[1, 0] = -1         # all of one
    bt[2, 2] = 1 << 30    # the last key of one: its rows see the rest
    bt[3, 0] = -7
    want = L.absorbed(L.values(pool), L.values(q), rs, lens, bt, SCALE)
    o, lse, err = run(H, pool, bt, lens, rs, q)
    assert err == H.DEV_BAD_PAGE
    check((o, lse), want, dtype, 320)
    assert (o[rs[1]:rs[2]] == 0).all() and (lse[rs[1]:rs[2]] == -np.inf).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_bad_lengths(H, dtype):
    lens, counts = [100, 200, 5, 300], [2, 9, 7, 1]
    rng, pool, bt, rs, q = latent_case(36, dtype, lens, counts, 16, 512)
    lens_bad = [100, 200, 3, 300]  # more rows than keys
    o, lse, err = run(H, pool, bt, lens_bad, rs, q, max_n=8)  # and more rows than declared
    assert err == H.DEV_BAD_LENGTH
    good = np.r_[rs[0]:rs[1], rs[3]:rs[4]]
    want = L.absorbed(L.values(pool), L.values(q), rs, lens, bt, SCALE)
    check((o[good], lse[good]), tuple(x[good] for x in want), dtype, 576)
    assert (o[rs[1]:rs[3]] == 9).all() and (lse[rs[1]:rs[3]] == 9).all()
    o, lse, err = run(H, pool, bt, lens, rs, q, max_t=250)  # more keys than declared
    assert err == H.DEV_BAD_LENGTH and (o[rs[3]:] == 9).all() and (o[:rs[3]] != 9).any()


def test_nan_and_inf(H):
    """A NaN in a query or a key gives NaN in the rows that see it and no others."""
    lens, counts = [200, 200], [3, 1]
    rng, pool, bt, rs, q = latent_case(37, "bf16", lens, counts, 16, 512)
    q[1, 5, 40] = 0x7FC0
    pool[bt[1, 1], 3, 575] = 0x7FC0  # sequence 1, the rotated part of key 67
    o, lse, err = run(H, pool, bt, lens, rs, q)
    assert err == 0
    nan = np.zeros((4, 16), bool)
    nan[1, 5], nan[3] = True, True
    assert (np.isnan(lse) == nan).all() and (np.isnan(o).any(-1) == nan).all()


def test_pool_beyond_32_bit_offsets(H):
    """Pages whose bytes and elements lie beyond 2^32 and 2^31."""
    import torch

    pages, lens = 60000, [200, 65]
    rng = np.random.default_rng(38)
    k = torch.zeros((pages, 1, 64, 576), dtype=torch.bfloat16, device="cuda")
    bt = np.array([[pages - 1, 3, pages - 9, 58254], [pages - 2, 7, -1, -1]], np.int32)
    vals = rng.standard_normal((6, 64, 576))
    used = bt[bt >= 0]
    raws = T.bf16_round(vals)
    for i, p in enumerate(used):
        k[int(p), 0] = T.device(raws[i])
    small = {int(p): i for i, p in enumerate(used)}
    bt_small = np.array([[small[int(p)] if p >= 0 else -1 for p in row] for row in bt], np.int32)
    rs = T.starts([2, 1])
    q = T.bf16_round(rng.standard_normal((3, 16, 576)))
    want = L.absorbed(T.widen(raws), T.widen(q), rs, lens, bt_small, SCALE)
    kv = H.KV(k=k, v=None, block_table=T.device(bt), seq_len=T.device(np.array(lens, np.int32)))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = H.hs2_latent_chunk(T.device(q), T.device(rs), kv, SCALE, 2, max_t=200, dev_err=err)
    assert int(err.item()) == 0
    check((o.double().cpu().numpy(), lse.cpu().numpy()), want, "bf16", 576)


def test_workspace_of_a_larger_call_suffices(H):
    import torch

    kv = H.KV(k=torch.zeros((4, 1, 64, 576), dtype=torch.bfloat16, device="cuda"), v=None,
              block_table=torch.zeros((3, 4), dtype=torch.int32, device="cuda"),
              seq_len=torch.ones(3, dtype=torch.int32, device="cuda"))
    for Hq in (1, 16, 128):
        big = H.hs2_latent_chunk_workspace(64, Hq, kv, 40, 256)
        for n, mn, mt in ((64, 40, 256), (63, 40, 256), (64, 1, 256), (64, 3, 100), (2, 2, 2), (1, 1, 1), (64, 8, 256)):
            assert H.hs2_latent_chunk_workspace(n, Hq, kv, mn, mt) <= big
    for Hq in (1, 16):
        big = H.hs2_latent_prefill_workspace(64, Hq, 3, 40, 256)
        for n, mn, mt in ((64, 40, 256), (1, 1, 1), (64, 1, 256), (30, 30, 30)):
            assert H.hs2_latent_prefill_workspace(n, Hq, 3, mn, mt) <= big


def test_graph_and_streams(H):
    """Captured and replayed with new values in place, and on a side stream, bit for bit as eager."""
    import torch

    lens, counts = [700, 64, 1, 300], [1, 2, 1, 5]
    rng, pool, bt, rs, q = latent_case(39, "bf16", lens, counts, 32, 512)
    kv, dq, drs = latent_kv(H, pool, bt, lens), T.device(q), T.device(rs)
    n = q.shape[0]
    out = (torch.zeros((n, 32, 512), device="cuda"), torch.zeros((n, 32), device="cuda"))
    ws = torch.empty(H.hs2_latent_chunk_workspace(n, 32, kv, 5, 700), dtype=torch.uint8, device="cuda")
    call = lambda: H.hs2_latent_chunk(dq, drs, kv, SCALE, 5, max_t=700, out=out, workspace=ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    dq.copy_(torch.randn_like(dq.float()).to(torch.bfloat16))
    kv.seq_len.copy_(torch.tensor([600, 64, 1, 299], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    got = [x.clone() for x in out]
    eager = H.hs2_latent_chunk(dq, drs, kv, SCALE, 5, max_t=700)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    on_side = H.hs2_latent_chunk(dq, drs, kv, SCALE, 5, max_t=700, stream=side)
    torch.cuda.synchronize()
    for a, b, c in zip(got, eager, on_side):
        assert torch.equal(a, b) and torch.equal(b, c)


@pytest.mark.parametrize("Hq,top", [(16, 200), (128, 200), (16, 3000), (128, 3000)])
def test_graphs_of_few_rows(H, Hq, top):
    """Two graphs of calls that plan in their blocks, in one workspace and replayed in turn while the lengths
    move, so that other units are cut each time."""
    import torch

    lens, counts = [top, 64, 1, top // 2 + 3], [1, 1, 0, 1]
    rng, pool, bt, rs, q = latent_case(54, "bf16", lens, counts, Hq, 256)
    n = q.shape[0]
    size = 0
    calls = []
    for seqs in (4, 2):  # all, and the first two with one row
        kv = latent_kv(H, pool, bt[:seqs], lens[:seqs])
        rows = T.device(q[:int(rs[seqs])].copy())
        calls.append((kv, rows, T.device(rs[:seqs + 1].copy())))
        size = max(size, H.hs2_latent_chunk_workspace(n, Hq, kv, 1, top))
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    graphs = []
    for kv, rows, drs in calls:
        out = torch.zeros((rows.shape[0], Hq, 256), device="cuda"), torch.zeros((rows.shape[0], Hq), device="cuda")
        run_it = lambda: H.hs2_latent_chunk(rows, drs, kv, SCALE, 1, max_t=top, out=out, workspace=ws)  # noqa: B023, E731
        run_it()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run_it()
        graphs.append((g, out))
    for now in ([top, 64, 1, top // 2 + 3], [1, 1, 1, 130], [top - 129, 20, 1, 64], [top, 63, 0, 2]):
        for kv, _, _ in calls:
            kv.seq_len.copy_(torch.tensor(now[:kv.seq_len.numel()], dtype=torch.int32))
        for g, _ in graphs * 2:
            g.replay()
        torch.cuda.synchronize()
        for (kv, rows, drs), (_, out) in zip(calls, graphs):
            seqs = kv.seq_len.numel()
            want = L.absorbed(L.values(pool), L.values(q[:rows.shape[0]]), rs[:seqs + 1], now[:seqs], bt[:seqs], SCALE)
            check((out[0].double().cpu().numpy(), out[1].cpu().numpy()), want, "bf16", 320)


def test_more_sequences_than_threads(H):
    """1100 sequences: the plan takes them 1024 at a time, and as many units."""
    lens = [1 + (i * 37) % 150 for i in range(1100)]
    counts = [0 if i % 7 == 3 else 1 for i in range(1100)]
    rng, pool, bt, rs, q = latent_case(40, "bf16", lens, counts, 4, 256)
    want = L.absorbed(L.values(pool), L.values(q), rs, lens, bt, SCALE)
    o, lse, err = run(H, pool, bt, lens, rs, q)
    assert err == 0
    check((o, lse), want, "bf16", 320)
    rng, rs, ks, q, kv, r = expanded_case(40, "bf16", counts, lens, 2)
    want = want_expanded(rs, ks, q, kv, r)
    o, lse, err = run_expanded(H, rs, ks, q, kv, r)
    assert err == 0
    check((o, lse), want, "bf16", 192)


@pytest.mark.parametrize("Hq", [16, 128])
def test_two_calls_at_once(H, Hq):
    """Two streams, a workspace each; and one after another in one workspace with other sizes."""
    import torch

    cases = [latent_case(48 + i, "bf16", lens, counts, Hq, 512) + (lens,) for i, (lens, counts) in
             enumerate((([3000, 500], [2, 1]), ([129] * 30, [1] * 30)))]
    ins = [(T.device(q), T.device(rs), latent_kv(H, pool, bt, lens), int(np.diff(rs).max()), max(lens))
           for rng, pool, bt, rs, q, lens in cases]
    alone = [H.hs2_latent_chunk(q, rs, kv, SCALE, mn, max_t=mt) for q, rs, kv, mn, mt in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    got = [[] for _ in ins]
    for _ in range(5):
        for i, (q, rs, kv, mn, mt) in enumerate(ins):
            got[i].append(H.hs2_latent_chunk(q, rs, kv, SCALE, mn, max_t=mt, stream=streams[i]))
    torch.cuda.synchronize()
    size = max(H.hs2_latent_chunk_workspace(q.shape[0], Hq, kv, mn, mt) for q, rs, kv, mn, mt in ins)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        for i, (q, rs, kv, mn, mt) in enumerate(ins):
            got[i].append(H.hs2_latent_chunk(q, rs, kv, SCALE, mn, max_t=mt, workspace=ws))
    torch.cuda.synchronize()
    for want, runs in zip(alone, got):
        for x in runs:
            assert torch.equal(x[0], want[0]) and torch.equal(x[1], want[1])


def spread(batch, top, low=1):
    """Lengths from low to top, in no order, the longest somewhere in the middle."""
    lens = [low + (top - low) * ((i * 7919 + 13) % 101) // 101 for i in range(batch)]
    lens[batch // 2] = top
    return lens


# What decides who plans: at most 32 sequences, 512 keys (expanded 1024), 16 units a block (of a pair of
# blocks: 76 pairs; else 152 blocks, with a unit more for each sequence); or at most 128 sequences of up to 64
# rows (pairs: 32 of up to 128). Batches and lengths on both sides.
@pytest.mark.parametrize("batch,top,tokens,Hq", [(32, 256, 1, 64), (33, 256, 1, 64), (32, 257, 2, 16), (33, 257, 2, 16),
                                                 (32, 512, 1, 32), (33, 512, 1, 32), (32, 513, 1, 128), (1, 512, 1, 128),
                                                 (32, 300, 37, 128), (32, 300, 38, 128), (40, 1300, 25, 16),
                                                 (150, 2000, 9, 16), (60, 900, 2, 64), (128, 2000, 1, 16),
                                                 (129, 2000, 1, 16), (64, 5000, 4, 32), (5, 3100, 1, 128), (128, 257, 4, 16),
                                                 (32, 2000, 1, 128), (33, 2000, 1, 128), (32, 900, 8, 16), (33, 900, 8, 16),
                                                 (100, 9000, 16, 1), (3, 700, 9, 16)])
def test_who_plans(H, batch, top, tokens, Hq):
    lens = spread(batch, top)
    counts = [0 if i % 9 == 4 else min(t, tokens) for i, t in enumerate(lens)]
    rng, pool, bt, rs, q = latent_case(50, "bf16", lens, counts, Hq, 256, first=1, extra=1)
    pool = poison(pool, bt, lens)
    want = L.absorbed(L.values(pool), L.values(q), rs, lens, bt, SCALE)
    o, lse, err = run(H, pool, bt, lens, rs, q, max_n=tokens)
    assert err == 0
    check((o, lse), want, "bf16", 320, rows=slice(rs[0], rs[-1]))
    for outside in (slice(0, rs[0]), slice(rs[-1], None)):
        assert (o[outside] == 9).all() and (lse[outside] == 9).all()
    again = run(H, pool, bt, lens, rs, q, max_n=tokens)
    assert (o == again[0]).all() and (lse == again[1]).all()


@pytest.mark.parametrize("Hq,top,more", [(16, 300, 9), (128, 300, 9), (8, 2900, 9), (128, 2900, 1), (1, 2900, 9)])
def test_bad_books_where_blocks_plan(H, Hq, top, more):
    """As test_bad_lengths and test_bad_pages where a block finds its units or its range itself."""
    lens, counts = [100, 200, 5, top, 0, 64], [min(2, more), more, min(4, more), 1, 0, 1]
    rng, pool, bt, rs, q = latent_case(51, "bf16", lens, counts, Hq, 512)
    bt[0, 0], bt[5, 0] = len(pool), -1
    want = L.absorbed(L.values(pool), L.values(q), rs, lens, bt, SCALE)
    # rows 9 > 8, 4 > 3; of single tokens: keys beyond max_t, none
    bad = [100, 200, 3, top, 0, 64] if more > 1 else [100, top + 1, 0, top, 0, 64]
    o, lse, err = run(H, pool, bt, bad, rs, q, max_n=min(8, more), max_t=top)
    assert err == H.DEV_BAD_LENGTH | H.DEV_BAD_PAGE
    good = np.r_[rs[0]:rs[1], rs[3]:rs[6]]
    check((o[good], lse[good]), tuple(x[good] for x in want), "bf16", 576)
    assert (o[rs[1]:rs[3]] == 9).all() and (lse[rs[1]:rs[3]] == 9).all()
    assert (o[rs[5]:] == 0).all() and (lse[rs[5]:] == -np.inf).all()
    falling = rs.copy()
    falling[2] = rs[1] - 1  # rows of two sequences at once: nobody's are computed
    o, lse, err = run(H, pool, bt, lens, falling, q, max_n=more)
    assert err == H.DEV_BAD_LENGTH and (o == 9).all() and (lse == 9).all()
    beyond = rs.copy()
    beyond[6] += 1  # rows that do not exist
    o, lse, err = run(H, pool, bt, lens, beyond, q, max_n=max(more, 2), max_t=top)
    assert err & H.DEV_BAD_LENGTH and (o[rs[5]:] == 9).all() and (o[rs[1]:rs[2]] != 9).any()


def test_workspace_grows_with_the_call(H):
    """Whoever plans: more rows, more rows of a sequence or more keys never need less."""
    import torch

    for batch in (1, 32, 33, 64, 128, 129):
        kv = H.KV(k=torch.zeros((1, 1, 64, 576), dtype=torch.bfloat16, device="cuda"), v=None,
                  block_table=torch.zeros((batch, 2000), dtype=torch.int32, device="cuda"),
                  seq_len=torch.ones(batch, dtype=torch.int32, device="cuda"))
        for Hq in (1, 16, 64, 128):
            def size(n, mn, mt):
                return H.hs2_latent_chunk_workspace(n, Hq, kv, mn, mt)
            steps = [(16, 64), (64, 256), (256, 512), (512, 513), (513, 100000)]
            for n in (1, 16, 128, 4000):
                for mn in (1, 2, 8, 9):
                    for lo, hi in steps:
                        assert size(n, mn, lo) <= size(n, mn, hi)
                    for mt in (64, 256, 512, 100000):
                        assert size(n, mn, mt) <= size(n + 1, mn, mt) and size(n, mn, mt) <= size(n, mn + 1, mt)


@pytest.mark.parametrize("tiles", [1023, 1024])
def test_longest_whole_units(H, tiles):
    """160 single tokens over up to 131072 keys, every page the same one: the softmax of its 64 keys, and
    lse log(pages) more. The sums are of 128 * tiles terms in fp32, each addition off by at most 2^-24 of
    the sum so far."""
    import torch

    pages, Hq, batch = 2 * tiles, 16, 160
    rng = np.random.default_rng(52)
    page = T.bf16_round(rng.standard_normal((1, 64, 320)))
    q = T.bf16_round(rng.standard_normal((batch, Hq, 320)))
    ro, rlse, mag = L.absorbed(T.widen(page), T.widen(q), T.starts([1] * batch), [64] * batch, np.zeros((batch, 1), int), SCALE)
    kv = H.KV(k=T.device(page[:, None]), v=None, block_table=torch.zeros((batch, pages), dtype=torch.int32, device="cuda"),
              seq_len=torch.full((batch,), 64 * pages, dtype=torch.int32, device="cuda"))
    o, lse = H.hs2_latent_chunk(T.device(q), T.device(T.starts([1] * batch)), kv, SCALE, 1, max_t=64 * pages)
    slack = 128 * tiles * 2.0 ** -24
    assert np.abs(lse.cpu().numpy() - rlse - np.log(pages)).max() <= slack + lse_tol(320)
    assert (np.abs(o.double().cpu().numpy() - ro) <= (2.0 ** -8 + 2 * lse_tol(320) + 2 * slack) * mag + 1e-6).all()


# ---------------------------------------------------------------------------- expanded
def expanded_case(seed, dtype, counts, keys, Hq, first=0, extra=0, key_first=0, key_extra=0):
    rng = np.random.default_rng(seed)
    rs, ks = T.starts(counts, first), T.starts(keys, key_first)
    nk = int(ks[-1]) + key_extra
    q = L.raw(rng.standard_normal((int(rs[-1]) + extra, Hq, 192)), dtype)
    kv = L.raw(rng.standard_normal((nk, Hq, 256)), dtype)
    r = L.raw(rng.standard_normal((nk, 64)), dtype)
    return rng, rs, ks, q, kv, r


def run_expanded(H, rs, ks, q, kv, r, scale=SCALE, o_dtype=None, max_n=None, max_t=None, **kw):
    import torch

    o_dtype = o_dtype or torch.float32
    n, Hq, _ = q.shape
    out = torch.full((n, Hq, 128), 9.0, device="cuda", dtype=o_dtype), torch.full((n, Hq), 9.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    d = T.device(kv)
    H.hs2_latent_prefill(T.device(q), d[..., :128], T.device(r), d[..., 128:], T.device(rs), T.device(ks), scale,
                         max_n if max_n is not None else int(np.diff(rs).max()),
                         max_t if max_t is not None else int(np.diff(ks).max()), o_dtype=o_dtype, out=out, dev_err=err, **kw)
    torch.cuda.synchronize()
    return out[0].double().cpu().numpy(), out[1].cpu().numpy(), int(err.item())


def want_expanded(rs, ks, q, kv, r):
    kv = L.values(kv)
    return L.expanded(L.values(q), kv[..., :128], L.values(r), kv[..., 128:], rs, ks, SCALE)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Hq", [1, 3, 8, 16])
def test_expanded_ragged(H, dtype, Hq):
    counts, keys = [1, 130, 64, 0, 37, 65, 1, 5], [1, 130, 200, 9, 300, 65, 128, 133]
    rng, rs, ks, q, kv, r = expanded_case(41, dtype, counts, keys, Hq, first=1, extra=2, key_first=2, key_extra=3)
    # what no sequence has, before, behind and (no rows: key 395 on) between, may be anything
    for x in (kv, r):
        x[:2] = x[ks[-1]:] = x[ks[3]:ks[4]] = 0x7FC0 if dtype == "bf16" else np.nan
    want = want_expanded(rs, ks, q, np.nan_to_num(kv) if dtype == "f32" else np.where(kv == 0x7FC0, 0, kv).astype(np.uint16),
                         np.nan_to_num(r) if dtype == "f32" else np.where(r == 0x7FC0, 0, r).astype(np.uint16))
    o, lse, err = run_expanded(H, rs, ks, q, kv, r)
    assert err == 0
    check((o, lse), want, dtype, 192, rows=slice(rs[0], rs[-1]))
    for outside in (slice(0, rs[0]), slice(rs[-1], None)):
        assert (o[outside] == 9).all() and (lse[outside] == 9).all()


@pytest.mark.parametrize("counts,keys,Hq", [([1000], [1000], 2), ([3, 700], [2000, 700], 4), ([1] * 200, [70] * 200, 2),
                                            ([257, 256, 255], [257, 300, 511], 3), ([129, 128, 127, 1], [129, 128, 127, 900], 2),
                                            ([40], [3000], 16)])
def test_expanded_long(H, counts, keys, Hq):
    import torch

    rng, rs, ks, q, kv, r = expanded_case(42, "bf16", counts, keys, Hq)
    want = want_expanded(rs, ks, q, kv, r)
    o, lse, err = run_expanded(H, rs, ks, q, kv, r, o_dtype=torch.bfloat16)
    assert err == 0
    check((o, lse), want, "bf16", 192, o_bf16=True)


@pytest.mark.parametrize("order", ["rising", "falling"])
def test_expanded_logits_that_grow(H, order):
    counts, keys = [300, 5], [700, 300]
    rng, rs, ks, q, kv, r = expanded_case(43, "bf16", counts, keys, 2)
    qv, rv = L.values(q).astype(np.float32), L.values(r).astype(np.float32)
    qv[..., 128:136] = 4.0
    for b, t in enumerate(keys):
        s = np.arange(t)
        rv[ks[b]:ks[b + 1], :8] = ((s if order == "rising" else t - s) / t * 300)[:, None]
    q, r = L.raw(qv, "bf16"), L.raw(rv, "bf16")
    ro, rlse, mag = want_expanded(rs, ks, q, kv, r)
    o, lse, err = run_expanded(H, rs, ks, q, kv, r)
    assert err == 0
    slack = 192 * 2.0 ** -23 * (32 * 300 * SCALE + 30)
    assert (np.abs(lse - rlse) <= slack + 1e-3).all()
    assert (np.abs(o - ro) <= (2.0 ** -8 + 2 * slack) * mag + 1e-6).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_expanded_bad_lengths(H, dtype):
    counts, keys = [2, 9, 7, 1], [100, 200, 5, 300]  # sequence 2: fewer keys than rows
    rng, rs, ks, q, kv, r = expanded_case(44, dtype, counts, keys, 2)
    o, lse, err = run_expanded(H, rs, ks, q, kv, r, max_n=8)
    assert err == H.DEV_BAD_LENGTH
    good = np.r_[rs[0]:rs[1], rs[3]:rs[4]]
    ks2 = ks.copy()
    kvv = L.values(kv)
    parts = [L.expanded(L.values(q)[rs[b]:rs[b + 1]], kvv[ks[b]:ks[b + 1], :, :128], L.values(r)[ks[b]:ks[b + 1]],
                        kvv[ks[b]:ks[b + 1], :, 128:], [0, counts[b]], [0, keys[b]], SCALE) for b in (0, 3)]
    want = tuple(np.concatenate(x) for x in zip(*parts))
    check((o[good], lse[good]), want, dtype, 192)
    assert (o[rs[1]:rs[3]] == 9).all()
    ks2[-1] += 50  # keys that do not exist
    o, lse, err = run_expanded(H, rs, ks2, q, kv, r, max_n=9, max_t=350)
    assert err == H.DEV_BAD_LENGTH and (o[rs[3]:] == 9).all()
    falling = ks.copy()
    falling[1] = 400
    assert run_expanded(H, rs, falling, q, kv, r, max_n=9, max_t=400)[2] == H.DEV_BAD_LENGTH


def test_expanded_strides(H):
    """K, V and r as slices of wider arrays, heads outermost, and one head of several."""
    import torch

    counts, keys, Hq = [70, 3], [200, 131], 4
    rng, rs, ks, q, kv, r = expanded_case(45, "bf16", counts, keys, Hq)
    want = want_expanded(rs, ks, q, kv, r)
    d, dr, dq = T.device(kv), T.device(r), T.device(q)
    nk = d.shape[0]
    wide = torch.full((nk, 64 + 8), float("nan"), device="cuda", dtype=torch.bfloat16)
    wide[:, :64] = dr
    k_heads = d[..., :128].transpose(0, 1).contiguous().transpose(0, 1)  # [n][H] over [H][n] memory
    v_pad = torch.full((nk, Hq, 136), float("nan"), device="cuda", dtype=torch.bfloat16)
    v_pad[..., :128] = d[..., 128:]
    o, lse = H.hs2_latent_prefill(dq, k_heads, wide[:, :64], v_pad[..., :128], T.device(rs), T.device(ks), SCALE, 70, 200)
    check((o.double().cpu().numpy(), lse.cpu().numpy()), want, "bf16", 192)
    one = tuple(x[:, 2:3] for x in want)
    o, lse = H.hs2_latent_prefill(dq[:, 2:3].contiguous(), d[:, 2:3, :128], dr, d[:, 2:3, 128:], T.device(rs),
                                  T.device(ks), SCALE, 70, 200)
    check((o.double().cpu().numpy(), lse.cpu().numpy()), one, "bf16", 192)


def test_expanded_graph(H):
    import torch

    counts, keys = [300, 1, 65], [300, 500, 80]
    rng, rs, ks, q, kv, r = expanded_case(46, "bf16", counts, keys, 4)
    dq, d, dr, drs, dks = T.device(q), T.device(kv), T.device(r), T.device(rs), T.device(ks)
    n = q.shape[0]
    out = torch.zeros((n, 4, 128), device="cuda"), torch.zeros((n, 4), device="cuda")
    ws = torch.empty(H.hs2_latent_prefill_workspace(n, 4, 3, 300, 500), dtype=torch.uint8, device="cuda")
    call = lambda: H.hs2_latent_prefill(dq, d[..., :128], dr, d[..., 128:], drs, dks, SCALE, 300, 500, out=out,  # noqa: E731
                                        workspace=ws)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    dq.mul_(0.5)
    g.replay()
    torch.cuda.synchronize()
    got = [x.clone() for x in out]
    eager = H.hs2_latent_prefill(dq, d[..., :128], dr, d[..., 128:], drs, dks, SCALE, 300, 500)
    for a, b in zip(got, eager):
        assert torch.equal(a, b)


@pytest.mark.parametrize("batch,top,tokens,Hq", [(32, 1024, 70, 4), (33, 1024, 70, 4), (32, 1025, 70, 4), (31, 512, 300, 3),
                                                 (33, 512, 300, 3), (32, 200, 48, 64), (32, 200, 56, 64), (36, 1500, 30, 8),
                                                 (70, 1500, 40, 16), (3, 1024, 1, 1)])
def test_expanded_who_plans(H, batch, top, tokens, Hq):
    """As test_who_plans; 64 heads of 32 sequences are 16 units a block up to 1536 rows."""
    keys = spread(batch, top, low=56 if Hq == 64 else 1)
    counts = [0 if Hq != 64 and i % 9 == 4 else min(t, tokens) for i, t in enumerate(keys)]
    rng, rs, ks, q, kv, r = expanded_case(53, "bf16", counts, keys, Hq, first=1, extra=1)
    want = want_expanded(rs, ks, q, kv, r)
    o, lse, err = run_expanded(H, rs, ks, q, kv, r, max_n=tokens)
    assert err == 0
    check((o, lse), want, "bf16", 192, rows=slice(rs[0], rs[-1]))
    for outside in (slice(0, rs[0]), slice(rs[-1], None)):
        assert (o[outside] == 9).all() and (lse[outside] == 9).all()
    again = run_expanded(H, rs, ks, q, kv, r, max_n=tokens)
    assert (o == again[0]).all() and (lse == again[1]).all()


# ---------------------------------------------------------------------------- together
def test_write_read_expand_attend(H):
    """A prompt and then tokens as a model runs them: latents appended with rotation, the prompt through
    the expanded form, the tokens through the absorbed one; both are the attention over R(p) r and
    the expansion W c. Each path's inputs are rounded to bf16 in its own places (latents expanded:
    k, v; queries absorbed: q W): off by 2^-8 of the logits' and values' terms."""
    import torch

    rng = np.random.default_rng(47)
    Hq, dc, lens0, new = 16, 512, [150, 64, 1], [1, 3, 2]
    W = rng.standard_normal((Hq, dc, 256)) / np.sqrt(dc)
    table = L.rot_table(400, 64)
    dW, dt = torch.from_numpy(W).cuda().float(), T.device(table)
    pages = 3 * 4
    pool = torch.full((pages, 1, 64, dc + 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    books = H.Pages.make(pages)
    bt = torch.full((3, 4), -1, dtype=torch.int32, device="cuda")
    sl = torch.zeros(3, dtype=torch.int32, device="cuda")
    kv = H.KV(k=pool, v=None, block_table=bt, seq_len=sl)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    all_c, all_r = [], []
    for step, counts in enumerate((lens0, new)):
        n = sum(counts)
        rs = T.starts(counts)
        lens = lens0 if step == 0 else [a + b for a, b in zip(lens0, new)]
        c, r = T.bf16_round(rng.standard_normal((n, dc))), T.bf16_round(rng.standard_normal((n, 64)))
        q = T.bf16_round(rng.standard_normal((n, Hq, 192)))
        dq, drs = T.device(q), T.device(rs)
        H.hs2_pages_grow(books, bt, sl, T.device(np.array(counts, np.int32)), dev_err=err)
        H.hs2_latent_write(kv, T.device(c), T.device(r), drs, dt, q=dq[..., 128:], q_out=dq[..., 128:], dev_err=err)
        all_c.append(c), all_r.append(r)
        rows, pos = L.positions(rs, lens)
        qv = T.widen(q)
        qv[rows] = np.concatenate([qv[rows][..., :128], T.widen(T.bf16_round(L.rotate(
            T.widen(q)[rows][..., 128:], pos, table, True)))], -1)
        assert np.array_equal(T.widen(T.host(dq)), qv)
        # the whole sequences, as they are in the cache
        ks = T.starts(lens)
        cc, rr = H.hs2_latent_read(kv, T.device(ks), int(ks[-1]), dev_err=err)
        seq_c = [T.widen(all_c[0][b0:b1]) for b0, b1 in zip(T.starts(lens0)[:-1], T.starts(lens0)[1:])]
        seq_r = [T.widen(all_r[0][b0:b1]) for b0, b1 in zip(T.starts(lens0)[:-1], T.starts(lens0)[1:])]
        if step:
            seq_c = [np.concatenate([a, T.widen(c)[rs[b]:rs[b + 1]]]) for b, a in enumerate(seq_c)]
            seq_r = [np.concatenate([a, T.widen(r)[rs[b]:rs[b + 1]]]) for b, a in enumerate(seq_r)]
        turned = np.concatenate([L.rotate(x[:, None], np.arange(len(x)), table, True)[:, 0] for x in seq_r])
        assert np.array_equal(T.widen(T.host(cc)), np.concatenate(seq_c))
        assert np.array_equal(T.widen(T.host(rr)), T.widen(T.bf16_round(turned)))
        full_kv = np.einsum("kc,hcd->khd", np.concatenate(seq_c), W)
        ro, rlse, mag = L.expanded(qv, full_kv[..., :128], T.widen(T.host(rr)), full_kv[..., 128:], rs, ks, SCALE)
        if step == 0:
            e = torch.einsum("kc,hcd->khd", cc.float(), dW).to(torch.bfloat16)
            o, lse = H.hs2_latent_prefill(dq, e[..., :128], rr, e[..., 128:], drs, T.device(ks), SCALE, max(counts), max(lens),
                                          dev_err=err)
            o = o.double().cpu().numpy()
        else:
            ql = torch.cat((torch.einsum("nhd,hcd->nhc", dq[..., :128].float(), dW[..., :128]).to(torch.bfloat16),
                            dq[..., 128:]), -1)
            ol, lse = H.hs2_latent_chunk(ql, drs, kv, SCALE, max(counts), dev_err=err)
            o = np.einsum("nhc,hcd->nhd", ol.double().cpu().numpy(), W[..., 128:])
        assert int(err.item()) == 0
        # logits: 128 (512) rounded factors, 2^-8 |q k| each, against sum |q k| scale < 12 (36): the
        # expanded form's off by 0.05 at most, the absorbed one's q W likewise per latent channel
        logit = 2.0 ** -8 * SCALE * (192 * 0.87 if step == 0 else 512 * 0.87)
        assert np.abs(lse.cpu().numpy() - rlse).max() <= logit
        assert (np.abs(o - ro) <= (2 * logit + 2.0 ** -7) * mag + 2.0 ** -7 * np.abs(ro).max()).all()
    # branches share the latents' pages; compaction moves them
    keep = kv.seq_len.clone()
    child_bt, child_len = H.hs2_pages_fork(books, [kv], T.device(np.array([0, 2], np.int32)), dev_err=err)
    child = H.KV(k=pool, v=None, block_table=child_bt, seq_len=child_len)
    ks = T.starts([int(keep[0]), int(keep[2])])
    a = H.hs2_latent_read(child, T.device(ks), int(ks[-1]), dev_err=err)
    full = T.starts([int(x) for x in keep])
    b = H.hs2_latent_read(kv, T.device(full), int(full[-1]), dev_err=err)
    for x, y in zip(a, b):
        assert torch.equal(x, torch.cat((y[full[0]:full[1]], y[full[2]:full[3]])))
    H.hs2_pages_free(books, child_bt, child_len, T.device(np.array([1, 1], np.int32)), dev_err=err)
    H.hs2_pages_free(books, bt[1:2].contiguous(), sl[1:2].contiguous(), T.device(np.array([1], np.int32)), dev_err=err)
    left = H.KV(k=pool, v=None, block_table=bt[[0, 2]].contiguous(), seq_len=sl[[0, 2]].contiguous())
    H.hs2_pages_compact(books, [left], dev_err=err)
    c2 = H.hs2_latent_read(left, T.device(ks), int(ks[-1]), dev_err=err)
    for x, y in zip(a, c2):
        assert torch.equal(x, y)
    assert int(err.item()) == 0
