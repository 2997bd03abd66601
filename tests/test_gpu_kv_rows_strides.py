"""K and V rows that lie differently: a tensor of its own and a slice of a wider one, single rows."""
import numpy as np
import pytest

import cache_testutil as T
from test_gpu_kv_rows import H, check_pools, row_values  # noqa: F401

pytestmark = pytest.mark.gpu


def laid(x, wide):
    """A device copy of the rows; wide: as a slice of rows that hold more."""
    import torch

    t = T.device(x)
    if not wide:
        return t
    n, h, d = t.shape
    big = torch.full((n, h * d + 48), 3.0, device="cuda").to(t.dtype)
    s = big[:, 16:16 + h * d].unflatten(1, (h, d))
    s.copy_(t)
    return s


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8", "fp4"])
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("kw,vw", [(False, True), (True, False), (True, True)])
def test_rows_of_different_strides(H, dtype, n, kw, vw):  # noqa: F811
    import torch

    rng = np.random.default_rng(16)
    lens = [n + 30, 9]
    c = T.make_cache(rng, dtype, 5, 2, 64, scale=1.0)
    bt = T.make_table(rng, lens, 5)
    rs = T.starts([n, 0])
    kv = T.device_cache(H, c, bt, lens)
    r, pg, ln = T.places(rs, lens, bt)
    dev, want = {}, c
    for side, wide in (("k", kw), ("v", vw)):
        raw, val = row_values(rng, n, 2, 64, "bf16")
        dev[side] = laid(raw, wide)
        want = T.write_rows(want, val, side, r, pg, ln)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    H.hs2_kv_write(kv, dev["k"], dev["v"], T.device(rs), dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    check_pools(kv, c, want)
    out = tuple(laid(np.zeros((n, 2, 64), np.float32), wide) for wide in (kw, vw))
    H.hs2_kv_read(kv, T.device(rs), n, out=out)
    k, v = H.hs2_kv_read(kv, T.device(rs), n)
    assert torch.equal(out[0], k) and torch.equal(out[1], v)
    assert (out[0].abs().sum() > 0) and (out[1].abs().sum() > 0)


def test_one_head_of_any_head_stride(H):  # noqa: F811
    """With one KV head, and with one row, the strides that no element is reached by do not matter."""
    import torch

    rng = np.random.default_rng(17)
    c = T.make_cache(rng, "bf16", 3, 1, 64)
    bt = T.make_table(rng, [50], 3)
    x = T.device(T.bf16_round(rng.standard_normal((50, 64)).astype(np.float32)))
    a, b = T.device_cache(H, c, bt, [50]), T.device_cache(H, c, bt, [50])
    rs = T.device(T.starts([50]))
    H.hs2_kv_write(a, x[:, None], x[:, None], rs)
    H.hs2_kv_write(b, x.as_strided((50, 1, 64), (64, 7, 1)), x[:, None], rs)
    assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v)
    one = T.device(T.starts([1]))
    for kv in (a, b):
        kv.seq_len = T.device(np.array([3], np.int32))
    H.hs2_kv_write(a, x[:1, None], x[:1, None], one)
    H.hs2_kv_write(b, x.as_strided((1, 1, 64), (999, 5, 1)), x[:1, None], one)
    assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v)


def test_strides_that_cannot_be_passed_are_refused_before_anything_is_written(H):  # noqa: F811
    """V rows off 16 bytes, or closer together than a row: refused, and K is not written either."""
    import torch

    rng = np.random.default_rng(18)
    c = T.make_cache(rng, "bf16", 3, 1, 64)
    bt = T.make_table(rng, [50], 3)
    kv = T.device_cache(H, c, bt, [50])
    k = torch.ones((50, 1, 64), device="cuda", dtype=torch.bfloat16)
    flat = torch.ones(50 * 80, device="cuda", dtype=torch.bfloat16)
    rs = T.device(T.starts([50]))
    for v in (flat.as_strided((50, 1, 64), (76, 64, 1)), flat[4:].as_strided((50, 1, 64), (72, 64, 1)),
              flat.as_strided((50, 1, 64), (32, 64, 1)), flat.as_strided((50, 1, 64), (0, 64, 1)), k.float(),
              flat.as_strided((50, 1, 64), (64, 64, 2))[:25]):
        with pytest.raises(H.HS2Error):
            H.hs2_kv_write(kv, k, v, rs)
    torch.cuda.synchronize()
    check_pools(kv, c, c)
