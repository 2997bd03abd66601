"""Attention of query chunks over FP8 and FP4 caches, on each of the ways a call can take: which
kernels run follows from the sizes that the caller declares (the most rows and keys of a sequence),
so the same batch is run with declared sizes that lead to each. Tolerances as in the tests of
hs2_fa_chunk: 128 * 2^-23 * 12 for a logit, and a weight's rounding to 16 bits times sum p |v| / Z."""
import numpy as np
import pytest

import cache_testutil as T
from test_gpu_chunk import H, LSE_TOL, case, check, poison, run  # noqa: F401

pytestmark = pytest.mark.gpu

LENS, COUNTS = [300, 65, 700, 40, 129, 0], [290, 1, 33, 40, 0, 0]
# (max_n, max_t): few rows times keys; more, with little to expand; much to expand
ROUTES = {"small": (290, 700), "expanded": (8192, 8192), "both": (131072, 131072)}


def routed(seed, dtype, d, route, Hq=16, Hkv=2):
    """The batch with a table as wide as the declared length; no entry behind a sequence's pages may
    be looked at, so they are out of range."""
    rng, c, bt, rs, qraw, qval = case(seed, dtype, LENS, COUNTS, Hq, Hkv, d, first=2, extra=1)
    max_n, max_t = ROUTES[route]
    wide = np.full((len(LENS), max(max_t // 64, bt.shape[1])), 10 ** 9, np.int32)
    for b, t in enumerate(LENS):
        n = -(-t // 64)
        wide[b, :n] = bt[b, :n]
    return rng, c, wide, rs, qraw, qval, dict(max_n=max_n, max_t=max_t)


@pytest.mark.parametrize("dtype", ["fp8", "fp4"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("route", ["small", "expanded", "both"])
@pytest.mark.parametrize("w,sink,obf", [(0, False, False), (50, True, True), (128, False, False), (0, True, True)])
def test_routes(H, dtype, d, route, w, sink, obf):  # noqa: F811
    import torch

    rng, c, bt, rs, qraw, qval, top = routed(41, dtype, d, route)
    c = poison(c, bt, LENS)
    s = (rng.standard_normal(16) * 3).astype(np.float32) if sink else None
    if sink:
        s[3] = -np.inf
    want = T.attend(c, qval, rs, LENS, bt, d ** -0.5, w, s)
    o, lse, err = run(H, c, bt, LENS, rs, qraw, d ** -0.5, w, s, o_dtype=torch.bfloat16 if obf else None, **top)
    assert err == 0
    check((o, lse), want, dtype, o_bf16=obf, rows=slice(rs[0], rs[-1]))
    for outside in (slice(0, rs[0]), slice(rs[-1], None)):
        assert (o[outside] == 9).all() and (lse[outside] == 9).all()


@pytest.mark.parametrize("dtype", ["fp8", "fp4"])
@pytest.mark.parametrize("route", ["small", "expanded", "both"])
def test_routes_with_extreme_scales_and_missing_pages(H, dtype, route):  # noqa: F811
    rng, c, bt, rs, qraw, qval, top = routed(42, dtype, 128, route)
    for b in (0, 2):  # logits that grow along the keys
        n = -(-LENS[b] // 64)
        c["k_scale"][bt[b, :n]] *= np.linspace(0.1, 6, n, dtype=np.float32)[:, None]
    c["v_scale"][bt[2, 1]] *= np.float32(2.0 ** 20)
    c["v_scale"][bt[2, 3]] = 0
    c["v_scale"][bt[0, 1]] *= np.float32(2.0 ** -20)
    c["v_scale"][bt[0, 0]] *= -1
    c["k_scale"][bt[2, 4]] *= -1
    bt[0, 2], bt[2, 5], bt[3, 0] = -1, c["num_pages"], -9
    ro, rlse, mag = T.attend(c, qval, rs, LENS, bt, 128 ** -0.5)
    o, lse, err = run(H, c, bt, LENS, rs, qraw, 128 ** -0.5, **top)
    assert err == H.DEV_BAD_PAGE
    rows = slice(rs[0], rs[-1])
    # 6 times the logits' size, so 6 times their fp32 errors
    assert (np.abs(o - ro) <= (2.0 ** -8 + 12 * LSE_TOL) * mag + 1e-6)[rows].all()
    fin = np.isfinite(rlse[rows])
    assert (np.isfinite(lse[rows]) == fin).all()
    assert np.abs(lse[rows][fin] - rlse[rows][fin]).max() <= 6 * LSE_TOL
    assert (o[rs[3]:rs[4]] == 0).all() and np.isneginf(lse[rs[3]:rs[4]]).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("route", ["small", "expanded"])
@pytest.mark.parametrize("e", [-60, -18, 16, 60])
def test_query_magnitudes(H, dtype, route, e):  # noqa: F811
    """Queries far from 1, `scale` the other way: a power of two changes no rounding on the way."""
    rng, c, bt, rs, qraw, qval, top = routed(43, dtype, 128, route)
    q = np.ldexp(T.widen(qraw), e)
    want = T.attend(c, q, rs, LENS, bt, float(np.ldexp(0.09, -e)))
    o, lse, err = run(H, c, bt, LENS, rs, T.bf16_round(q.astype(np.float32)), float(np.ldexp(0.09, -e)), **top)
    assert err == 0
    check((o, lse), want, dtype, rows=slice(rs[0], rs[-1]))
    del rng, qval


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "fp4"])
def test_many_sequences(H, dtype):  # noqa: F811
    """More sequences than the planning kernel's threads, most of them of one token."""
    rng = np.random.default_rng(44)
    lens = [int(x) for x in rng.integers(1, 200, 1500)]
    counts = [1 if i % 7 else 0 for i in range(1500)]
    lens[700], counts[700] = 400, 350
    r, c, bt, rs, qraw, qval = case(45, dtype, lens, counts, 8, 1, 64)
    want = T.attend(c, qval, rs, lens, bt, 0.125)
    o, lse, err = run(H, c, bt, lens, rs, qraw, 0.125)
    assert err == 0
    check((o, lse), want, dtype)
    del r


def test_two_graphs_share_a_workspace(H):  # noqa: F811
    """Two captured calls with one workspace, replayed in turn on one stream, each leave their own
    results."""
    import torch

    made = []
    nb = 0
    for seed, route in ((46, "small"), (47, "both")):
        rng, c, bt, rs, qraw, qval, top = routed(seed, "fp4", 128, route)
        kv = T.device_cache(H, c, bt, LENS)
        nb = max(nb, H.hs2_fa_chunk_workspace(len(qraw), 16, kv, top["max_n"], top["max_t"]))
        made.append((T.device(qraw), T.device(rs), kv, top, rs, T.attend(c, qval, rs, LENS, bt, 0.1)))
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    outs, graphs = [], []
    for q, rs, kv, top, _, _ in made:
        outs.append((torch.empty(q.shape, device="cuda"), torch.empty(q.shape[:2], device="cuda")))
        call = lambda: H.hs2_fa_chunk(q, rs, kv, 0.1, top["max_n"], max_t=top["max_t"], workspace=ws, out=outs[-1])  # noqa: E731
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            call()
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
    for _ in range(2):
        for g, o in zip(graphs, outs):
            o[0].fill_(9), o[1].fill_(9)
            g.replay()
    torch.cuda.synchronize()
    for (o, lse), m in zip(outs, made):
        check((o.double().cpu().numpy(), lse.cpu().numpy()), m[5], "fp4", rows=slice(m[4][0], m[4][-1]))
