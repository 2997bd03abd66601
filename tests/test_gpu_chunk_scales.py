"""Attention of query chunks over FP8 and FP4 caches whose V scales are small, large or far from one
another, on each of the ways a call can take.

Tolerance: the weights are rounded to 16 bits (at most 2^-8 of each), the logits' errors come to
2 * LSE_TOL (as in the tests of hs2_fa_chunk), and fp32 sums over a few thousand keys to less; all of
that is relative to sum p |v| / Z, so there is no absolute term: an output that is lost shows at
every scale. Weights far below a row's largest contribution count in full here, as N(0, 1) logits
keep them within 2^-12 of it."""
import numpy as np
import pytest

import cache_testutil as T
from test_gpu_chunk import H, LSE_TOL, case, run  # noqa: F401
from test_gpu_chunk_routes import ROUTES

pytestmark = pytest.mark.gpu

REL = 2.0 ** -8 + 2 * LSE_TOL
# declared rows and keys of a sequence that lead to each way, for two or three sequences, one KV head, d = 64
ONE_HEAD = {"small": None, "expanded": 131072, "both": 1 << 20}


def one_head(route, counts, lens):
    top = ONE_HEAD[route]
    return (max(counts), max(lens)) if top is None else (top, top)


def check_relative(got, want, rows, lse_tol=LSE_TOL, rel=REL, lost=0):
    (o, lse), (ro, rlse, mag) = got, want
    worst = (np.abs(o - ro) - rel * mag - lost)[rows]
    assert worst.max() <= 0, (np.abs(o - ro)[rows] / np.maximum(mag[rows], 1e-300)).max()
    fin = np.isfinite(rlse[rows])
    assert (np.isfinite(lse[rows]) == fin).all()
    assert np.abs(lse[rows][fin] - rlse[rows][fin]).max(initial=0) <= lse_tol


def below_range(c, qval, rs, lens, bt, scale, w):
    """What f16 weights lose where a row sees scales far apart and the larger ones' codes happen to be
    zero in a channel, so that the channel's sum p |v| is the smaller ones' alone.
    The kernel for few rows multiplies codes by p S in f16 units in which the row's largest p S is at
    least 2^6 (its reference puts it there and moves only upwards past 2^14). A value below f16's
    normal range is off by half its step, 2^-25, so a key's p S by at most 2^-31 of the row's largest,
    and a channel by at most 2^-31 * max(p S) / Z * sum |code|, of which max(p S) <= sum p S. Rows that do
    not see the large scales have small ones here, and the term is nothing beside their sum p |v|."""
    one = dict(c, v=np.full_like(c["v"], 0x38 if c["dtype"] == "fp8" else 0x22))  # V of ones
    if c["dtype"] == "fp4":
        one["v_sf"] = np.full_like(c["v_sf"], 0x38)
    weight = T.attend(one, qval, rs, lens, bt, scale, w)[2]
    codes = T.attend(dict(c, v_scale=np.ones_like(c["v_scale"])), 0 * qval, rs, lens, bt, scale, w)[2]
    seen = np.concatenate([t - (e - b) + np.arange(e - b) + 1 for t, b, e in zip(lens, rs, rs[1:])])
    seen = np.minimum(seen, w) if w else seen
    return 2.0 ** -31 * weight * codes * seen[:, None, None]


def widened(bt, lens, max_t):
    wide = np.full((len(lens), max(max_t // 64, bt.shape[1])), 10 ** 9, np.int32)
    for b, t in enumerate(lens):
        wide[b, :-(-t // 64)] = bt[b, :-(-t // 64)]
    return wide


@pytest.mark.parametrize("dtype", ["fp8", "fp4"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("route", ["small", "expanded", "both"])
@pytest.mark.parametrize("e", [-60, -50, -40, -30, -24, 0, 40, 60])
def test_every_v_scale_alike(H, dtype, d, route, e):  # noqa: F811
    """All V scales near 2^e: sequences within one page, of odd and even page counts, and with an
    entry out of range among their pages."""
    lens, counts = [300, 1, 64, 65, 129, 700, 40], [290, 1, 3, 65, 2, 33, 0]
    rng, c, bt, rs, qraw, qval = case(81, dtype, lens, counts, 16, 2, d, first=1, extra=1)
    c["v_scale"] = np.ldexp(c["v_scale"] * np.float32(16), e)
    max_n, max_t = ROUTES[route]
    bt = widened(bt, lens, max_t)
    bt[5, 2], bt[5, 7] = -1, c["num_pages"]
    want = T.attend(c, qval, rs, lens, bt, d ** -0.5)
    o, lse, err = run(H, c, bt, lens, rs, qraw, d ** -0.5, max_n=max_n, max_t=max_t)
    assert err == H.DEV_BAD_PAGE
    check_relative((o, lse), want, slice(rs[0], rs[-1]))
    del rng


@pytest.mark.parametrize("dtype", ["fp8", "fp4"])
@pytest.mark.parametrize("route", ["small", "expanded", "both"])
@pytest.mark.parametrize("far", [20, 40, 60])
def test_pages_of_larger_scale_that_a_row_does_not_see(H, dtype, route, far):  # noqa: F811
    """Pages whose scale is 2^far times the others': later keys of the same chunk, and keys before a
    window that share a page or a tile with it."""
    lens, counts = [330, 70, 129], [180, 20, 100]
    max_n, max_t = one_head(route, counts, lens)
    for w, pages in ((0, (5, 1, 2)), (40, (1, 0, 0))):
        rng, c, bt, rs, qraw, qval = case(82, dtype, lens, counts, 8, 1, 64)
        for b, j in enumerate(pages):
            c["v_scale"][bt[b, j]] *= np.float32(2.0 ** far)
        bt = widened(bt, lens, max_t)
        want = T.attend(c, qval, rs, lens, bt, 0.125, w)
        o, lse, err = run(H, c, bt, lens, rs, qraw, 0.125, w, max_n=max_n, max_t=max_t)
        assert err == 0
        check_relative((o, lse), want, slice(None), lost=below_range(c, qval, rs, lens, bt, 0.125, w))
        del rng


@pytest.mark.parametrize("dtype", ["fp8", "fp4"])
@pytest.mark.parametrize("route", ["small", "expanded", "both"])
@pytest.mark.parametrize("n", [2, 60, 200])
def test_pages_of_larger_scale_that_weigh_nothing(H, dtype, route, n):  # noqa: F811
    """The weight lies on pages whose scale is 2^-50 of their neighbours', whose keys have logits
    some 300 lower; with a scale of zero among them, and sinks."""
    lens, counts = [n + 460, n], [n, n]
    max_n, max_t = one_head(route, counts, lens)
    rng, c, bt, rs, qraw, qval = case(83, dtype, lens, counts, 8, 1, 64)
    qraw, qval = qraw & np.uint16(0x7FFF), np.abs(qval)
    for j in (0, 3, 5):
        p = bt[0, j]
        c["k"][p] |= np.uint8(0x80 if dtype == "fp8" else 0x88)
        c["k_scale"][p] *= 64
        c["v_scale"][p] *= np.float32(2.0 ** 50)
    c["v_scale"][bt[0, 2]] = 0
    bt = widened(bt, lens, max_t)
    s = rng.standard_normal(8).astype(np.float32)
    for sink in (None, s):
        want = T.attend(c, qval, rs, lens, bt, 0.125, sink=sink)
        o, lse, err = run(H, c, bt, lens, rs, qraw, 0.125, sink=sink, max_n=max_n, max_t=max_t)
        assert err == 0
        check_relative((o, lse), want, slice(None))


@pytest.mark.parametrize("dtype", ["fp8", "fp4"])
@pytest.mark.parametrize("scale", [0.0, 2.0 ** -60])
def test_rows_that_see_one_scale_only(H, dtype, scale):  # noqa: F811
    """Every V page of scale zero gives zeros and the right lse; the smallest scale gives its values."""
    lens, counts = [64, 1, 130, 300], [2, 1, 1, 200]
    rng, c, bt, rs, qraw, qval = case(84, dtype, lens, counts, 8, 1, 128)
    c["v_scale"][:] = scale
    for top in ({}, dict(max_n=8192, max_t=131072)):
        wide = widened(bt, lens, top.get("max_t", 0))
        want = T.attend(c, qval, rs, lens, wide, 0.1)
        o, lse, err = run(H, c, wide, lens, rs, qraw, 0.1, **top)
        assert err == 0
        check_relative((o, lse), want, slice(None))
        assert scale or (o == 0).all()
    del rng


@pytest.mark.parametrize("dtype", ["fp8", "fp4"])
def test_long_ranges(H, dtype):  # noqa: F811
    """More than 16 tiles to a CTA, so that page entries and scales are fetched in several blocks: scales
    that fall along the keys, entries out of range, odd page counts."""
    lens, counts = [64 * 1702 + 3] * 3, [1, 2, 4]
    rng, c, bt, rs, qraw, qval = case(85, dtype, lens, counts, 8, 1, 64)
    for b in range(3):
        n = -(-lens[b] // 64)
        c["v_scale"][bt[b, :n]] *= np.exp2(-np.arange(n, dtype=np.float32) / 64)[:, None]
        bt[b, 37::61] = -1
    want = T.attend(c, qval, rs, lens, bt, 0.125, w=0)
    o, lse, err = run(H, c, bt, lens, rs, qraw, 0.125)
    assert err == H.DEV_BAD_PAGE
    # sums of 1e5 weights in fp32, each addition off by 2^-24 of the sum at most and a CTA's part some
    # 2200 keys of 128 threads: below 2e-4 in all
    check_relative((o, lse), want, slice(None), lse_tol=2 * LSE_TOL, rel=REL + 2e-4)
    del rng


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("n", [2, 300])
def test_logits_up_to_the_documented_size(H, dtype, n):  # noqa: F811
    """Logits of nearly 2^26: finite, lse within the logits' own fp32 errors (a sum of d = 128 products in
    fp32: 128 * 2^-23 * scale * sum |q k|), and where the largest leads by more than twice those, the
    row is that key's V up to a weight's rounding to 16 bits."""
    t = 700
    rng, c, bt, rs, qraw, qval = case(86, dtype, [t], [n], 8, 1, 128)
    page, line = bt[0, np.arange(t) // 64], np.arange(t) % 64
    k, v = (T.values(c, side, page, 0, line) for side in ("k", "v"))
    x = np.einsum("nhd,td->nht", qval, k)
    scale = float(np.float32(0.99 * 2.0 ** 26 / np.abs(x).max()))
    seen = np.arange(t) <= t - n + np.arange(n)[:, None, None]
    x = np.where(seen, scale * x, -np.inf)
    off = 128 * 2.0 ** -23 * scale * np.where(seen, np.einsum("nhd,td->nht", np.abs(qval), np.abs(k)), 0).max(-1)
    o, lse, err = run(H, c, bt, [t], rs, qraw, scale)
    assert err == 0 and np.isfinite(o).all()
    assert (np.abs(lse - x.max(-1)) <= off + 10).all()  # (log of the number of keys: below 10)
    top = np.sort(x, -1)
    clear = top[..., -1] - top[..., -2] > 2 * off + 40
    assert clear.mean() > 0.9
    want = v[x.argmax(-1)][clear]
    assert (np.abs(o[clear] - want) <= 2.0 ** -8 * np.abs(want) + 1e-12).all()
    del rng
