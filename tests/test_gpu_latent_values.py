"""Latent attention over values that are not finite: every route of either form. A NaN in a key or a
query, or a logit of +inf, gives NaN in the rows that see it and in no others; a logit of -inf is a
weight of 0. Tolerances as in test_gpu_latent."""
import numpy as np
import pytest

import latent_testutil as L
from test_gpu_latent import (H, SCALE, check, expanded_case, latent_case, run, run_expanded)  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu

KINDS = {"nan": np.nan, "plus": np.inf, "minus": -np.inf}


def put(x, at, value, dtype):
    """x[at] = value in x's type."""
    x[at] = value if dtype == "f32" else L.raw(np.full((1,), value), "bf16")[0]


# (heads, lengths, tokens): a sequence that many blocks share (its parts merged), one of several units, short ones;
# 16, 32, 64 and 128 rows a unit; whole units that a plan hands out; blocks that plan themselves
SHAPES = [(16, [9000, 300, 7], [1, 1, 1]), (8, [2000, 700, 7], [30, 1, 3]), (32, [3000, 300, 7], [1, 2, 7]),
          (64, [3000, 300, 7], [1, 1, 1]), (128, [5000, 300, 7], [1, 1, 1]), (64, [1500, 130, 7], [40, 2, 5]),
          (128, [400, 130, 7], [3, 2, 5]), (4, [600] * 160, [1] * 160), (128, [256, 130, 7], [1, 1, 1])]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype,dc", [("bf16", 512), ("bf16", 256), ("f32", 256)])
@pytest.mark.parametrize("Hq,lens,counts", SHAPES)
def test_absorbed(H, kind, dtype, dc, Hq, lens, counts):  # noqa: F811
    """The last rotated channel is 1 in every query and not finite in a key about the middle, which the
    first of several rows of a sequence may not see, and in all keys of the last sequence."""
    rng, pool, bt, rs, q = latent_case(71, dtype, lens, counts, Hq, dc)
    put(q, (slice(None), slice(None), -1), 1.0, dtype)
    special = [(t - n // 2 - 1 if n > 1 else t // 2) for t, n in zip(lens, counts)]
    last = len(lens) - 1
    for b in {0, 1, last}:
        keys = np.arange(lens[b]) if b == last else np.array([special[b]])
        for s in keys:
            put(pool, (bt[b, s // 64], s % 64, -1), KINDS[kind], dtype)
    sees = np.zeros(len(q), bool)
    for b in {0, 1, last}:
        pos = lens[b] - counts[b] + np.arange(counts[b])
        sees[rs[b]:rs[b + 1]] = (pos >= special[b]) | (b == last)
    kv, qv = L.values(pool), L.values(q)
    if kind != "minus":
        kv = np.where(np.isfinite(kv), kv, 0)
    want = L.absorbed(kv, qv, rs, lens, bt, SCALE)
    o, lse, err = run(H, pool, bt, lens, rs, q)
    assert err == 0
    if kind == "minus":
        check((o, lse), want, dtype, dc + 64)
        assert (o[rs[last]:] == 0).all() and (lse[rs[last]:] == -np.inf).all()
    else:
        assert (np.isnan(lse) == sees[:, None]).all() and (np.isnan(o) == sees[:, None, None]).all()
        check((o[~sees], lse[~sees]), tuple(x[~sees] for x in want), dtype, dc + 64)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,lens,counts", [SHAPES[0], SHAPES[3], SHAPES[4], SHAPES[5]])
def test_absorbed_queries(H, dtype, Hq, lens, counts):  # noqa: F811
    """A NaN in one head's query: that row alone, not those beside it in its tile."""
    rng, pool, bt, rs, q = latent_case(72, dtype, lens, counts, Hq, 256)
    want = L.absorbed(L.values(pool), L.values(q), rs, lens, bt, SCALE)
    hit = np.zeros(q.shape[:2], bool)
    for r, h in ((0, 0), (0, Hq - 1), (len(q) - 1, Hq // 2)):
        put(q, (r, h, 33), np.nan, dtype)
        hit[r, h] = True
    o, lse, err = run(H, pool, bt, lens, rs, q)
    assert err == 0
    assert (np.isnan(lse) == hit).all() and (np.isnan(o) == hit[..., None]).all()
    check((o[~hit], lse[~hit]), tuple(x[~hit] for x in want), dtype, 320)


# a half or both, a unit that many blocks share, several units, whole units of a plan, blocks that plan themselves
EXPANDED = [(2, [3], [3000]), (2, [200, 5], [1500, 300]), (3, [700, 3], [700, 2000]), (2, [40] * 40, [1200] * 40), (4, [129, 37], [300, 90])]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("where", ["k", "r"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,counts,keys", EXPANDED)
def test_expanded(H, kind, where, dtype, Hq, counts, keys):  # noqa: F811
    """As test_absorbed; in k one head's logits alone, in r those of all heads."""
    rng, rs, ks, q, kv, r = expanded_case(73, dtype, counts, keys, Hq)
    put(q, (slice(None), slice(None), 5), 1.0, dtype)
    put(q, (slice(None), slice(None), 128 + 63), 1.0, dtype)
    last = len(keys) - 1
    special = [t - n // 2 - 1 if n > 1 else t // 2 for t, n in zip(keys, counts)]
    sees = np.zeros((len(q), Hq), bool)
    for b in {0, last}:
        s = slice(ks[b], ks[b + 1]) if b == last and b > 0 else ks[b] + special[b]
        if where == "k":
            put(kv, (s, Hq - 1, 5), KINDS[kind], dtype)
        else:
            put(r, (s, 63), KINDS[kind], dtype)
        pos = keys[b] - counts[b] + np.arange(counts[b])
        sees[rs[b]:rs[b + 1], Hq - 1 if where == "k" else slice(None)] = ((pos >= special[b]) | (b == last and b > 0))[
            (...,) if where == "k" else (..., None)]
    kvv, rv = L.values(kv), L.values(r)
    if kind != "minus":
        kvv, rv = np.where(np.isfinite(kvv), kvv, 0), np.where(np.isfinite(rv), rv, 0)
    want = L.expanded(L.values(q), kvv[..., :128], rv, kvv[..., 128:], rs, ks, SCALE)
    o, lse, err = run_expanded(H, rs, ks, q, kv, r)
    assert err == 0
    if kind == "minus":
        check((o, lse), want, dtype, 192)
        if last > 0:
            rows, head = slice(rs[last], None), Hq - 1
            assert (o[rows, head] == 0).all() and (lse[rows, head] == -np.inf).all()
    else:
        assert (np.isnan(lse) == sees).all() and (np.isnan(o) == sees[..., None]).all()
        check((o[~sees], lse[~sees]), tuple(x[~sees] for x in want), dtype, 192)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,counts,keys", EXPANDED)
def test_expanded_queries(H, dtype, Hq, counts, keys):  # noqa: F811
    rng, rs, ks, q, kv, r = expanded_case(74, dtype, counts, keys, Hq)
    kvv = L.values(kv)
    want = L.expanded(L.values(q), kvv[..., :128], L.values(r), kvv[..., 128:], rs, ks, SCALE)
    hit = np.zeros(q.shape[:2], bool)
    for row, h, ch in ((0, 0, 3), (1, Hq - 1, 130), (len(q) - 1, 1, 191)):
        put(q, (row, h, ch), np.nan, dtype)
        hit[row, h] = True
    o, lse, err = run_expanded(H, rs, ks, q, kv, r)
    assert err == 0
    assert (np.isnan(lse) == hit).all() and (np.isnan(o) == hit[..., None]).all()
    check((o[~hit], lse[~hit]), tuple(x[~hit] for x in want), dtype, 192)
