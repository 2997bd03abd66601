"""The paged-cache entry points reject bad arguments on the host, before any launch, and the
binding rejects tensors the library cannot take."""
import ctypes

import pytest

from top_hs2_fa_gb300 import build
from top_hs2_fa_gb300 import hs2 as H


@pytest.fixture(scope="module")
def lib():
    build.build()
    return H.load()


def _kv(**over):
    base = dict(k=16, v=32, block_table=48, seq_len=64, batch=2, num_pages=10, max_pages=5, page_size=64, Hkv=2,
                d=128, dtype=1)
    base.update(over)
    return H.hs2_kv(**base)


def _rows(call, kv, k=256, v=512, dt=1, stride=256, rs=1024, n=3):
    return call(ctypes.byref(kv), k, v, dt, stride, rs, n, None, None)


def test_rows_arguments(lib):
    for call in (lib.hs2_kv_write, lib.hs2_kv_read):
        for bad in (dict(k=0), dict(k=264), dict(v=0), dict(v=520), dict(dt=2), dict(dt=3), dict(dt=-1), dict(stride=248),
                    dict(stride=257), dict(stride=260), dict(rs=0), dict(n=-1)):
            assert _rows(call, _kv(), **bad) == -1, bad
        for over in (dict(page_size=32), dict(d=96), dict(dtype=2), dict(dtype=3, k_scale=64, v_scale=64), dict(k=17),
                     dict(v=40), dict(batch=0), dict(seq_len=0), dict(dtype=7)):
            assert _rows(call, _kv(**over)) == -1, over
        assert _rows(call, _kv(), n=0) == 0  # nothing to do, nothing launched


def _chunk(lib, kv, q=256, rs=512, n=4, max_n=3, Hq=8, max_t=300, w=0, scale=0.1, sink=None, o=1024, dt=0, ws=4096,
           wsb=1 << 40):
    return lib.hs2_fa_chunk(q, rs, n, max_n, Hq, ctypes.byref(kv), max_t, w, scale, sink, o, dt, None, ws, wsb, None, None)


def test_chunk_arguments(lib):
    for bad in (dict(q=0), dict(q=260), dict(rs=0), dict(n=-1), dict(max_n=-1), dict(max_n=301), dict(Hq=7), dict(Hq=0),
                dict(max_t=5 * 64 + 1), dict(w=-1), dict(scale=0.0), dict(scale=-0.1), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(o=0), dict(o=1028), dict(dt=2), dict(ws=0), dict(ws=4096 + 16), dict(wsb=8)):
        assert _chunk(lib, _kv(), **bad) == -1, bad
    assert _chunk(lib, _kv(), Hq=6) == -2
    assert _chunk(lib, _kv(Hkv=1), Hq=64) == -2
    for over in (dict(v=0), dict(d=96), dict(page_size=16), dict(dtype=2), dict(dtype=3, k_scale=64, v_scale=64)):
        assert _chunk(lib, _kv(**over)) == -1, over
    assert _chunk(lib, _kv(), n=0) == 0 and _chunk(lib, _kv(), max_n=0) == 0
    kv = _kv()
    assert lib.hs2_fa_chunk_workspace(4, 8, ctypes.byref(kv), 3, 300, 0) % 256 == 0
    assert lib.hs2_fa_chunk_workspace(4, 8, ctypes.byref(kv), 3, 300, 0) > 0
    assert lib.hs2_fa_chunk_workspace(-1, 8, ctypes.byref(kv), 3, 300, 0) == 0


def _pg(**over):
    base = dict(ref=16, free_list=32, n_free=48, num_pages=10)
    base.update(over)
    return H.hs2_pages(**base)


def test_pages_arguments(lib):
    grow = lambda p, t=64, n=80, new=96, b=2, mp=5: lib.hs2_pages_grow(  # noqa: E731
        ctypes.byref(p), t, n, new, b, mp, None, None)
    free = lambda p, t=64, n=80, d=96, b=2, mp=5: lib.hs2_pages_free(  # noqa: E731
        ctypes.byref(p), t, n, d, b, mp, None, None)
    for call in (grow, free):
        for over in (dict(ref=0), dict(free_list=0), dict(n_free=0), dict(num_pages=0)):
            assert call(_pg(**over)) == -1, over
        assert call(_pg(), t=0) == -1 and call(_pg(), n=0) == -1 and call(_pg(), b=-1) == -1 and call(_pg(), mp=0) == -1
        assert call(_pg(), mp=(1 << 20) + 1) == -2
        assert call(_pg(), b=0) == 0
    assert grow(_pg(), new=0) == -1 and free(_pg(), d=0) == -1


def test_fork_and_compact_arguments(lib):
    def fork(p, kvs, src=64, n=2, t=128, length=160):
        return lib.hs2_pages_fork(ctypes.byref(p), len(kvs), (H.hs2_kv * max(1, len(kvs)))(*kvs), src, n, t, length,
                                  None, None)

    def compact(p, kvs, ws=4096, wsb=1 << 20):
        return lib.hs2_pages_compact(ctypes.byref(p), len(kvs), (H.hs2_kv * max(1, len(kvs)))(*kvs), ws, wsb, None,
                                     None)

    for call in (fork, compact):
        assert call(_pg(), []) == -1
        assert call(_pg(), [_kv()] * 9) == -1
        assert call(_pg(num_pages=9), [_kv()]) == -1
        assert call(_pg(ref=0), [_kv()]) == -1
        for over in (dict(block_table=52), dict(seq_len=68), dict(batch=3), dict(max_pages=6), dict(num_pages=11),
                     dict(d=96), dict(k=17)):
            assert call(_pg(), [_kv(), _kv(**over)]) == -1, over
    assert fork(_pg(), [_kv()], src=0) == -1 and fork(_pg(), [_kv()], n=-1) == -1
    assert fork(_pg(), [_kv()], t=0) == -1 and fork(_pg(), [_kv()], length=0) == -1
    assert fork(_pg(), [_kv()], n=0) == 0
    p = _pg()
    assert lib.hs2_pages_compact_workspace(ctypes.byref(p)) >= 4 * 10
    assert compact(_pg(), [_kv()], ws=0) == -1 and compact(_pg(), [_kv()], ws=4100) == -1
    assert compact(_pg(), [_kv()], wsb=16) == -1


def test_binding_refuses_tensors_it_cannot_pass(lib):
    torch = pytest.importorskip("torch")
    kv = H.KV(k=torch.zeros(4, 2, 64, 64, dtype=torch.bfloat16), v=torch.zeros(4, 2, 64, 64, dtype=torch.bfloat16),
              block_table=torch.zeros(2, 2, dtype=torch.int32), seq_len=torch.ones(2, dtype=torch.int32))
    rows = torch.zeros(3, 2, 64)
    rs = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(H.HS2Error):  # host tensors
        H.hs2_kv_write(kv, rows, rows, rs)
    with pytest.raises(H.HS2Error):
        H.hs2_fa_chunk(torch.zeros(3, 4, 64, dtype=torch.bfloat16), rs, kv, 0.1, 1)
    with pytest.raises(H.HS2Error):
        H.hs2_fa_chunk(torch.zeros(3, 4, 64), rs, kv, 0.1, 1)  # float32 queries of a bf16 cache
    with pytest.raises(H.HS2Error):
        H.Pages(ref=torch.zeros(4), free_list=rs, n_free=rs).c()
    with pytest.raises(H.HS2Error):
        H.hs2_pages_grow(H.Pages.make(4, "cpu"), kv.block_table, kv.seq_len, rs)
