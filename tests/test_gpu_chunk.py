"""Attention of ragged query chunks over a paged cache, against the 64-bit form.

Tolerances, from the roundings on the way (u = half a step: bf16 2^-8, fp32 2^-24):
 lse  a logit is a sum of d exact products in fp32: off by at most d * 2^-23 * scale * sum |q k|
      (2^-23 an addition: round to nearest, or truncation on the tensor cores), which for N(0, 1)
      inputs stays below 128 * 2^-23 * 12 = 1.9e-4; exp2, log2 and the sums add a few 2^-22.
 o    the weights enter P.V rounded to 16 bits: off by u * sum p |v| / Z, plus the logits'
      errors, plus u |o| where o is bfloat16."""
import numpy as np
import pytest

import cache_testutil as T

pytestmark = pytest.mark.gpu
LSE_TOL = 3e-4


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


def case(seed, dtype, lens, counts, Hq, Hkv, d, first=0, extra=0, spare=2):
    rng = np.random.default_rng(seed)
    pages = sum(-(-max(t, 0) // 64) for t in lens) + spare
    c = T.make_cache(rng, dtype, pages, Hkv, d)
    bt = T.make_table(rng, lens, pages)
    rs = T.starts(counts, first)
    n = int(rs[-1]) + extra
    q = rng.standard_normal((n, Hq, d)).astype(np.float32)
    qraw = q if dtype == "f32" else T.bf16_round(q)
    qval = q.astype(np.float64) if dtype == "f32" else T.widen(qraw)
    return rng, c, bt, rs, qraw, qval


def poison(c, bt, lens):
    """NaN in every row that no sequence sees (behind its end, and in pages of nobody)."""
    seen = np.zeros((c["num_pages"], 64), bool)
    for b, t in enumerate(lens):
        for s in range(t):
            p = bt[b, s // 64]
            if 0 <= p < c["num_pages"]:
                seen[p, s % 64] = True
    page, line = np.nonzero(~seen)
    for side in ("k", "v"):
        if c["dtype"] == "f32":
            c[side][page, :, line] = np.nan
        elif c["dtype"] == "bf16":
            c[side][page, :, line] = 0x7FC0
        elif c["dtype"] == "fp8":
            c[side][page, :, line] = 0x7F
        else:
            c[side + "_sf"][page, :, line] = 0x7F
    return c


def run(H, c, bt, lens, rs, qraw, scale, w=0, sink=None, o_dtype=None, max_n=None, max_t=None, lse=True, **kw):
    import torch

    kv = T.device_cache(H, c, bt, lens)
    o_dtype = o_dtype or torch.float32
    n, Hq, d = qraw.shape
    out = (torch.full((n, Hq, d), 9.0, device="cuda", dtype=o_dtype),
           torch.full((n, Hq), 9.0, device="cuda") if lse else None)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    H.hs2_fa_chunk(T.device(qraw), T.device(rs), kv, scale, max_n if max_n is not None else int(np.diff(rs).max()),
                   max_t=max_t if max_t is not None else int(max(lens)), w=w,
                   sink=None if sink is None else T.device(sink), o_dtype=o_dtype, out=out, dev_err=err, **kw)
    torch.cuda.synchronize()
    return out[0].double().cpu().numpy(), out[1].cpu().numpy() if lse else None, int(err.item())


def check(got, want, dtype, o_bf16=False, rows=None):
    (o, lse), (ro, rlse, mag) = got, want
    rows = slice(None) if rows is None else rows
    u = 1e-5 if dtype == "f32" else 2.0 ** -8
    tol = (u + 2 * LSE_TOL) * mag + (2.0 ** -8 * np.abs(ro) if o_bf16 else 0) + 1e-6
    worst = (np.abs(o - ro) - tol)[rows]
    assert worst.size == 0 or worst.max() <= 0, (worst.max(), np.unravel_index(worst.argmax(), worst.shape))
    if lse is not None:
        fin = np.isfinite(rlse[rows])
        assert (np.isfinite(lse[rows]) == fin).all()
        assert np.abs(lse[rows][fin] - rlse[rows][fin]).max(initial=0) <= LSE_TOL * 1.0


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8", "fp4"])
@pytest.mark.parametrize("Hq,Hkv,d", [(8, 1, 128), (4, 4, 64), (32, 1, 128), (8, 2, 64), (32, 2, 128), (4, 2, 128)])
def test_ragged_heads(H, dtype, Hq, Hkv, d):
    lens, counts = [1, 130, 64, 300, 65, 7, 0], [1, 1, 64, 37, 0, 7, 0]
    rng, c, bt, rs, qraw, qval = case(21, dtype, lens, counts, Hq, Hkv, d, first=1, extra=2)
    c = poison(c, bt, lens)
    want = T.attend(c, qval, rs, lens, bt, d ** -0.5)
    o, lse, err = run(H, c, bt, lens, rs, qraw, d ** -0.5)
    assert err == 0
    inside = slice(rs[0], rs[-1])
    check((o, lse), want, dtype, rows=inside)
    for outside in (slice(0, rs[0]), slice(rs[-1], None)):  # rows of nobody stay as they were
        assert (o[outside] == 9).all() and (lse[outside] == 9).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8", "fp4"])
@pytest.mark.parametrize("w,sink", [(0, True), (1, False), (16, True), (64, False), (128, True), (1000, False)])
def test_window_and_sink(H, dtype, w, sink):
    import torch

    lens, counts = [500, 129, 1, 260], [300, 1, 1, 5]
    rng, c, bt, rs, qraw, qval = case(22, dtype, lens, counts, 8, 2, 64)
    s = (rng.standard_normal(8) * 3).astype(np.float32) if sink else None
    if sink:
        s[1], s[2] = -np.inf, 20.0
    want = T.attend(c, qval, rs, lens, bt, 0.125, w, s)
    o, lse, err = run(H, c, bt, lens, rs, qraw, 0.125, w, s, o_dtype=torch.bfloat16)
    assert err == 0
    check((o, lse), want, dtype, o_bf16=True)


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("counts,lens", [
    ([1] * 5, [2000, 63, 1, 4097, 640]), ([4] * 3, [1500, 4, 777]), ([16, 9], [900, 2050]),
    ([200], [1500]), ([700], [700]), ([513, 1, 2, 130], [1025, 3000, 66, 130])])
def test_longer(H, dtype, counts, lens):
    rng, c, bt, rs, qraw, qval = case(23, dtype, lens, counts, 16, 2, 128)
    c = poison(c, bt, lens)
    want = T.attend(c, qval, rs, lens, bt, 128 ** -0.5)
    o, lse, err = run(H, c, bt, lens, rs, qraw, 128 ** -0.5)
    assert err == 0
    check((o, lse), want, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("n", [1, 3, 40, 300])
def test_peaked_and_growing_logits(H, dtype, n):
    """Logits that grow along the keys (the running maximum moves all the time) and single keys
    that take nearly all the weight; slab scales that differ by 2^20 and one that is zero or
    negative."""
    lens, counts = [n + 500, n], [n, n]
    rng, c, bt, rs, qraw, qval = case(24, dtype, lens, counts, 8, 1, 128)
    if dtype == "bf16":
        ramp = np.linspace(0.1, 6, 64 * bt.shape[1])
        for j, p in enumerate(bt[0]):
            x = T.widen(c["k"][p]) * ramp[64 * j:64 * j + 64][None, :, None]
            c["k"][p] = T.bf16_round(x.astype(np.float32))
    else:
        c["k_scale"][bt[0]] *= np.linspace(0.1, 6, bt.shape[1], dtype=np.float32)[:, None]
        c["v_scale"][bt[0, 1]] *= np.float32(2.0 ** 20)
        c["v_scale"][bt[0, 2]] = 0
        c["v_scale"][bt[0, 3]] *= np.float32(2.0 ** -20)
        c["v_scale"][bt[0, 0]] *= -1
        c["k_scale"][bt[0, 4]] *= -1
    want = T.attend(c, qval, rs, lens, bt, 128 ** -0.5)
    o, lse, err = run(H, c, bt, lens, rs, qraw, 128 ** -0.5)
    assert err == 0
    ro, rlse, mag = want
    # 6 times the logits' size, so 6 times their fp32 errors
    tol = (2.0 ** -8 + 12 * LSE_TOL) * mag + 1e-6
    assert (np.abs(o - ro) <= tol).all()
    assert np.abs(lse - rlse).max() <= 6 * LSE_TOL


def test_bad_pages_are_left_out(H):
    import torch

    for dtype in ("f32", "bf16", "fp8", "fp4"):
        for n in (1, 150):
            lens, counts = [500, 64], [n, min(n, 64)]
            rng, c, bt, rs, qraw, qval = case(25, dtype, lens, counts, 8, 1, 64)
            bt[0, 2], bt[0, 5], bt[1, 0] = -1, c["num_pages"], -7
            want = T.attend(c, qval, rs, lens, bt, 0.125)
            o, lse, err = run(H, c, bt, lens, rs, qraw, 0.125)
            assert err == H.DEV_BAD_PAGE
            check((o, lse), want, dtype)
            assert (o[rs[1]:rs[2]] == 0).all() and np.isneginf(lse[rs[1]:rs[2]]).all()
    del torch


@pytest.mark.parametrize("dtype", ["f32", "fp4"])
@pytest.mark.parametrize("n", [2, 140])
def test_bad_sequences_are_flagged(H, dtype, n):
    """Sequences longer than the table, shorter than their rows, with more rows than max_n or rows
    beyond the buffer: flagged, their rows untouched; the others computed."""
    lens, counts = [300, n - 1, 5000, 200, 160], [n, n, n, n + 3, n]
    rng, c, bt, rs, qraw, qval = case(26, dtype, [300, 300, 300, 300, 160], counts, 8, 1, 64)
    want = T.attend(c, qval, rs, [300, 300, 300, 300, 160], bt, 0.125)
    qcut = qraw[:-1]  # the last sequence's last row lies behind the buffer
    o, lse, err = run(H, c, bt, lens, rs, qcut, 0.125, max_n=n, max_t=300)
    assert err == H.DEV_BAD_LENGTH
    check((o[:rs[1]], lse[:rs[1]]), tuple(x[:rs[1]] for x in want), dtype)
    assert (o[rs[1]:] == 9).all() and (lse[rs[1]:] == 9).all()


def test_without_lse_and_decode_parity(H):
    """lse may be left out; single tokens give what the framework's decode FA gives."""
    import torch

    lens = [700, 64, 1, 1500]
    for dtype in ("bf16", "fp8", "fp4"):
        rng, c, bt, rs, qraw, qval = case(27, dtype, lens, [1] * 4, 16, 2, 128)
        o, lse, err = run(H, c, bt, lens, rs, qraw, 0.09)
        o2, none, err2 = run(H, c, bt, lens, rs, qraw, 0.09, lse=False)
        assert err == err2 == 0 and none is None and np.array_equal(o, o2)
        kv = T.device_cache(H, c, bt, lens)
        fo, flse, _, _ = H.hs2_fa_select(T.device(qraw), kv, 0, 0, 0.09, max_t=1500)
        assert np.abs(fo.cpu().numpy() - o).max() <= 2e-2 and np.abs(flse.cpu().numpy() - lse).max() <= 2e-2
    del torch


def test_repeatable_and_reused_workspace(H):
    """The same call twice gives the same bits, and a workspace left dirty by another call does
    not matter."""
    import torch

    for counts, lens in (([1, 3, 2], [3000, 900, 40]), ([260, 1], [2000, 700])):
        rng, c, bt, rs, qraw, qval = case(28, "fp4", lens, counts, 8, 1, 128)
        kv = T.device_cache(H, c, bt, lens)
        nb = H.hs2_fa_chunk_workspace(len(qraw), 8, kv, max(counts), max(lens))
        ws = torch.full((nb,), 255, dtype=torch.uint8, device="cuda")
        q, drs = T.device(qraw), T.device(rs)
        a = [x.clone() for x in H.hs2_fa_chunk(q, drs, kv, 0.1, max(counts), max_t=max(lens), workspace=ws)]
        b = H.hs2_fa_chunk(q, drs, kv, 0.1, max(counts), max_t=max(lens), workspace=ws)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        check((a[0].double().cpu().numpy(), a[1].cpu().numpy()), T.attend(c, qval, rs, lens, bt, 0.1), "fp4")
