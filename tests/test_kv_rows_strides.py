"""What the binding passes on for rows of various strides (no launch: the library's entry is replaced)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from top_hs2_fa_gb300 import hs2 as H  # noqa: E402


@pytest.fixture
def calls(monkeypatch):
    got = []

    def entry(kv, k, v, dtype, stride, row_start, n, err, stream):
        c = ctypes.cast(kv, ctypes.POINTER(H.hs2_kv)).contents
        got.append(dict(pool=c.k, second=c.v, scale=c.k_scale, sf=c.k_sf, k=k, v=v, stride=stride, n=n))
        return 0

    class Lib:
        hs2_kv_write = staticmethod(entry)

    monkeypatch.setattr(H, "load", lambda: Lib)
    monkeypatch.setattr(H, "_launch_stream", lambda *a: 0)
    return got


def cache(Hkv):
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    return H.KV(k=u8(4, Hkv, 64, 32), v=u8(4, Hkv, 64, 32), block_table=torch.zeros(1, 2, dtype=torch.int32),
                seq_len=torch.ones(1, dtype=torch.int32), k_scale=torch.ones(4, Hkv), v_scale=torch.ones(4, Hkv),
                k_sf=u8(4, Hkv, 64, 4), v_sf=u8(4, Hkv, 64, 4))


START = torch.zeros(2, dtype=torch.int32)


def test_equal_strides_are_one_call(calls):
    kv, wide = cache(2), torch.zeros(5, 400)
    k, v = (wide[:, i:i + 128].unflatten(1, (2, 64)) for i in (16, 160))
    H.hs2_kv_write(kv, k, v, START)
    assert [(x["k"], x["v"], x["stride"], x["second"]) for x in calls] == [(k.data_ptr(), v.data_ptr(), 400, kv.v.data_ptr())]


def test_other_strides_are_a_call_a_side(calls):
    kv, wide = cache(2), torch.zeros(5, 400)
    k, v = torch.zeros(5, 2, 64), wide[:, 160:288].unflatten(1, (2, 64))
    H.hs2_kv_write(kv, k, v, START)
    assert [(x["pool"], x["scale"], x["sf"], x["k"], x["stride"]) for x in calls] == [
        (kv.k.data_ptr(), kv.k_scale.data_ptr(), kv.k_sf.data_ptr(), k.data_ptr(), 128),
        (kv.v.data_ptr(), kv.v_scale.data_ptr(), kv.v_sf.data_ptr(), v.data_ptr(), 400)]
    assert all(x["second"] is None and not x["v"] for x in calls)


def test_strides_that_reach_nothing_do_not_matter(calls):
    kv = cache(1)
    x = torch.zeros(64 * 5)
    H.hs2_kv_write(kv, x.as_strided((1, 1, 64), (7, 3, 1)), x.as_strided((1, 1, 64), (64, 64, 1)), START)
    H.hs2_kv_write(kv, x.as_strided((5, 1, 64), (64, 3, 1)), x.as_strided((5, 1, 64), (64, 64, 1)), START)
    assert [x["stride"] for x in calls] == [64, 64]


def test_refusals_come_before_any_call(calls):
    kv, k = cache(1), torch.zeros(5, 1, 64)
    flat = torch.zeros(600)
    for v in (flat.as_strided((5, 1, 64), (66, 64, 1)), flat[1:].as_strided((5, 1, 64), (68, 64, 1)),
              flat.as_strided((5, 1, 64), (32, 64, 1)), flat.as_strided((5, 1, 64), (0, 64, 1)),
              flat.as_strided((5, 1, 64), (68, 64, 2)), k.bfloat16(), k[:4], None):
        with pytest.raises(H.HS2Error):
            H.hs2_kv_write(kv, k, v, START)
    assert calls == []
