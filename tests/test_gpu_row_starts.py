"""Row starts that fall or point behind the rows: flagged on every route, rows of other sequences as they
should be."""
import numpy as np
import pytest

import cache_testutil as T
from test_gpu_chunk import H, case, check, run  # noqa: F401

pytestmark = pytest.mark.gpu

LENS = [200, 70, 90, 64]
# (starts, rows that a sequence owns on every reading of them, rows that may be owned)
FALLING = [([0, 10, 5, 20, 30], 30, 40), ([0, 30, 50, 40, 60], 30, 30), ([0, 100, 50, 60, 60], 30, 30),
           ([0, 10, 20, 60, 50], 20, 20)]
BEHIND = [([0, 10, 30, 31, 31], 30), ([0, 10, 10, 50, 50], 30), ([0, 30, 60, 60, 64], 30), ([-3, 5, 10, 12, 12], 12)]


def flags(H, call):  # noqa: F811
    import torch

    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    call(err)
    torch.cuda.synchronize()
    return int(err.item())


def owned(starts, n_rows, lens):
    """Rows of the sequences that are in order and lie within the rows."""
    rows = np.zeros(n_rows, bool)
    for b, t in enumerate(lens):
        lo, hi = starts[b], starts[b + 1]
        if 0 <= lo <= hi <= n_rows and hi - lo <= t:
            rows[lo:hi] = True
    return rows


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp4"])
@pytest.mark.parametrize("starts,n_rows", [(s, n) for s, n, _ in FALLING] + [(s, m) for s, _, m in FALLING] + BEHIND)
def test_rows_in_and_out(H, dtype, starts, n_rows):  # noqa: F811
    """hs2_kv_write and hs2_kv_read: flagged wherever in the starts the fault lies. Where no start
    falls, the other sequences' rows are written and read."""
    import torch

    rng = np.random.default_rng(91)
    c = T.make_cache(rng, dtype, 12, 1, 64, scale=1.0)
    bt = T.make_table(rng, LENS, 12)
    kv = T.device_cache(H, c, bt, LENS)
    x = rng.standard_normal((n_rows, 1, 64)).astype(np.float32)
    rows, drs = T.device(x), T.device(np.array(starts, np.int32))
    assert flags(H, lambda e: H.hs2_kv_write(kv, rows, rows, drs, dev_err=e)) == H.DEV_BAD_LENGTH
    out = tuple(torch.full((n_rows, 1, 64), 7.0, device="cuda") for _ in range(2))
    assert flags(H, lambda e: H.hs2_kv_read(kv, drs, n_rows, out=out, dev_err=e)) == H.DEV_BAD_LENGTH
    if (starts, n_rows) in BEHIND:
        own = owned(starts, n_rows, LENS)
        kept = [max(0, starts[b + 1] - starts[b]) if 0 <= starts[b] and starts[b + 1] <= n_rows else 0 for b in range(4)]
        r, pg, ln = [], [], []
        for b, n in enumerate(kept):
            for i in range(n):
                r.append(starts[b] + i), pg.append(bt[b, (LENS[b] - n + i) // 64]), ln.append((LENS[b] - n + i) % 64)
        want = c
        for side in ("k", "v"):
            want = T.write_rows(want, x.astype(np.float64), side, np.array(r, int), np.array(pg, int), np.array(ln, int))
        got = T.cache_arrays(kv, c)
        for name in got:
            np.testing.assert_array_equal(got[name], want[name], err_msg=name)
        assert (out[0].cpu().numpy()[~own] == 7).all() and (out[0].cpu().numpy()[own] != 7).any(-1).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp4"])
@pytest.mark.parametrize("starts,n_rows", [(s, n) for s, n, _ in FALLING] + [(s, m) for s, _, m in FALLING] + BEHIND)
def test_attention(H, dtype, starts, n_rows):  # noqa: F811
    """hs2_fa_chunk: flagged on every route. Rows of nobody stay as they were; float32 computes the
    rows of sequences that are in order, 16-bit and smaller caches compute none where a start falls."""
    rng, c, bt, rs, qraw, qval = case(92, dtype, LENS, [n_rows, 0, 0, 0], 8, 1, 64)
    o, lse, err = run(H, c, bt, LENS, np.array(starts, np.int32), qraw, 0.1, max_n=64, max_t=200)
    assert err == H.DEV_BAD_LENGTH
    falls = (np.diff(starts) < 0).any()
    own = owned(starts, n_rows, LENS) if dtype == "f32" or not falls else np.zeros(n_rows, bool)
    if falls and dtype == "f32":  # of rows that two sequences claim either may have them, or none
        claims = sum(np.isin(np.arange(n_rows), np.arange(max(0, starts[b]), max(0, starts[b + 1]))) for b in range(4))
        sure = claims == 0
    else:
        sure = ~own
    assert (o[sure] == 9).all() and (lse[sure] == 9).all()
    good = [b for b in range(4) if 0 <= starts[b] <= starts[b + 1] <= n_rows and starts[b + 1] - starts[b] <= LENS[b]]
    if falls:
        return
    for b in good:
        r0, r1 = starts[b], starts[b + 1]
        want = T.attend(c, qval[r0:r1], [0, r1 - r0], [LENS[b]], bt[b:b + 1], 0.1)
        check((o[r0:r1], lse[r0:r1]), want, dtype)
    del rng, rs


def test_float32_rows_of_falling_starts(H):  # noqa: F811
    """float32: with starts 0, 10, 5, 20, 30 the first ten rows are one sequence's and 20 to 30 another's
    on any reading; they are computed or left, never another sequence's values, and nobody's rows stay."""
    lens = [200, 70, 90, 64]
    rng, c, bt, rs, qraw, qval = case(93, "f32", lens, [40, 0, 0, 0], 8, 1, 64)
    starts = [0, 10, 5, 20, 30]
    o, lse, err = run(H, c, bt, lens, np.array(starts, np.int32), qraw, 0.1, max_n=16, max_t=200)
    assert err == H.DEV_BAD_LENGTH
    assert (o[30:] == 9).all() and (lse[30:] == 9).all()
    for r in range(30):
        wants = []
        for b in range(4):
            if starts[b] <= r < starts[b + 1]:
                n = starts[b + 1] - starts[b]
                q = np.repeat(qval[r:r + 1], n, 0)
                w = T.attend(c, q, [0, n], [lens[b]], bt[b:b + 1], 0.1)
                wants.append(w[0][r - starts[b]])
        left = (o[r] == 9).all()
        assert left or any(np.abs(o[r] - w).max() < 1e-4 for w in wants), r
    assert not (o[5:10] == 9).all() or not (o[20:30] == 9).all()
    del rng, rs
