"""The latent-attention and rotating entry points reject bad arguments on the host, before any launch,
and the binding rejects tensors the library cannot take."""
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


def _latent(**over):
    return _kv(**{**dict(v=0, Hkv=1, d=576), **over})


def _rot(**over):
    return H.hs2_rot(**{**dict(table=16, n_pos=100, dim=64, pairs=0), **over})


def _write_rot(lib, kv, rot, k=256, ks=256, v=512, vs=256, dt=1, rs=1024, n=3, q=2048, qs=512, Hq=4, qo=4096, qos=512):
    return lib.hs2_kv_write_rot(ctypes.byref(kv), k, ks, v, vs, dt, rs, n, ctypes.byref(rot) if rot else None, q, qs, Hq, qo,
                                qos, None, None)


def test_write_rot_arguments(lib):
    for bad in (dict(k=0), dict(k=264), dict(ks=248), dict(ks=257), dict(v=0), dict(v=520), dict(vs=255), dict(vs=128), dict(dt=2),
                dict(dt=-1), dict(rs=0), dict(n=-1), dict(q=0), dict(q=2056), dict(qs=511), dict(qs=504), dict(Hq=0),
                dict(Hq=-1), dict(qo=0), dict(qo=4104), dict(qos=504), dict(ks=1 << 32), dict(qs=1 << 32),
                dict(qo=2048, qos=520), dict(qo=2048, dt=0)):
        assert _write_rot(lib, _kv(), _rot(), **bad) == -1, bad
    for over in (dict(table=0), dict(table=24), dict(n_pos=0), dict(dim=0), dict(dim=16), dict(dim=48), dict(dim=160),
                 dict(pairs=2), dict(pairs=-1)):
        assert _write_rot(lib, _kv(), _rot(**over)) == -1, over
    assert _write_rot(lib, _kv(), None) == -1
    for over in (dict(page_size=32), dict(d=576), dict(dtype=2), dict(k=17), dict(v=40), dict(batch=0), dict(seq_len=0)):
        assert _write_rot(lib, _kv(**over), _rot()) == -1, over
    assert _write_rot(lib, _kv(), _rot(), n=0) == 0


def _latent_write(lib, kv, rot, c=256, cs=576, r=1280, rs=576, dt=1, start=1024, n=3, q=2048, qs=16 * 192 + 16, qh=192, Hq=16,
                  qo=4096, qos=16 * 576, qoh=576):
    return lib.hs2_latent_write(ctypes.byref(kv), c, cs, r, rs, dt, start, n, ctypes.byref(rot) if rot else None, q, qs, qh, Hq,
                                qo, qos, qoh, None, None)


def test_latent_rows_arguments(lib):
    for bad in (dict(c=0), dict(c=264), dict(cs=511), dict(cs=504), dict(r=0), dict(r=1288), dict(rs=56), dict(dt=2), dict(dt=9),
                dict(start=0), dict(n=-1), dict(q=0), dict(Hq=0), dict(Hq=-2), dict(qo=0), dict(qs=2000), dict(qh=63), dict(qh=56),
                dict(qoh=60), dict(qos=576), dict(qh=196), dict(q=4096, qo=4096), dict(cs=1 << 32)):
        assert _latent_write(lib, _latent(), _rot(), **bad) == -1, bad
    for over in (dict(dim=32), dict(dim=128), dict(table=0), dict(pairs=3), dict(n_pos=0)):
        assert _latent_write(lib, _latent(), _rot(**over)) == -1, over
    read = lambda kv, c=256, cs=512, r=1280, rs=64, dt=1, start=1024, n=3: lib.hs2_latent_read(  # noqa: E731
        ctypes.byref(kv), c, cs, r, rs, dt, start, n, None, None)
    for bad in (dict(c=0), dict(cs=508), dict(r=0), dict(rs=48), dict(dt=3), dict(start=0), dict(n=-1)):
        assert read(_latent(), **bad) == -1, bad
    for call in (lambda kv, **a: _latent_write(lib, kv, _rot(), **a), read):
        for over in (dict(v=32), dict(Hkv=2), dict(d=128), dict(d=512), dict(page_size=32), dict(k=0), dict(k=24), dict(batch=0),
                     dict(block_table=0)):
            assert call(_latent(**over)) == -1, over
        assert call(_latent(dtype=2)) == -2 and call(_latent(dtype=3)) == -2
        assert call(_latent(), n=0) == 0


def _chunk(lib, kv, q=256, rs=512, n=4, max_n=3, Hq=16, max_t=300, scale=0.1, o=1024, dt=0, ws=4096, wsb=1 << 40):
    return lib.hs2_latent_chunk(q, rs, n, max_n, Hq, ctypes.byref(kv), max_t, scale, o, dt, None, ws, wsb, None, None)


def test_latent_chunk_arguments(lib):
    for bad in (dict(q=0), dict(q=260), dict(rs=0), dict(n=-1), dict(max_n=-1), dict(max_n=301), dict(Hq=0), dict(max_t=321),
                dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(o=0), dict(o=1028), dict(dt=2), dict(ws=0),
                dict(ws=4096 + 16), dict(wsb=8)):
        assert _chunk(lib, _latent(), **bad) == -1, bad
    for Hq in (3, 24, 256):
        assert _chunk(lib, _latent(), Hq=Hq) == -2
    for over in (dict(v=32), dict(Hkv=2), dict(d=128), dict(d=512), dict(page_size=16)):
        assert _chunk(lib, _latent(**over)) == -1, over
    assert _chunk(lib, _latent(dtype=2)) == -2
    assert _chunk(lib, _latent(num_pages=1 << 25)) == -2  # 32-bit rows
    assert _chunk(lib, _latent(), n=0) == 0 and _chunk(lib, _latent(), max_n=0) == 0
    kv = _latent()
    assert lib.hs2_latent_chunk_workspace(4, 16, ctypes.byref(kv), 3, 300) > 0
    for bad in ((-1, 16, 3, 300), (4, 0, 3, 300), (4, 3, 3, 300), (4, 16, -1, 300), (4, 16, 3, -1)):
        assert lib.hs2_latent_chunk_workspace(*bad[:2], ctypes.byref(kv), *bad[2:]) == 0


def _keys(**over):
    return H.hs2_latent_keys(**{**dict(k=256, r=512, v=768, k_token=1024, k_head=256, r_token=64, v_token=1024, v_head=256,
                                       key_start=1024, n_keys=9, dtype=1), **over})


def _prefill(lib, keys, q=256, rs=512, n=4, max_n=3, Hq=4, batch=2, max_t=300, scale=0.1, o=1024, dt=0, ws=4096, wsb=1 << 40):
    return lib.hs2_latent_prefill(q, rs, n, max_n, Hq, batch, ctypes.byref(keys) if keys else None, max_t, scale, o, dt, None, ws,
                                  wsb, None, None)


def test_latent_prefill_arguments(lib):
    for bad in (dict(q=0), dict(q=260), dict(rs=0), dict(n=-1), dict(max_n=-1), dict(max_n=301), dict(Hq=0), dict(batch=0),
                dict(scale=-1.0), dict(scale=float("nan")), dict(o=0), dict(o=1028), dict(dt=3), dict(ws=0), dict(ws=4096 + 16),
                dict(wsb=8)):
        assert _prefill(lib, _keys(), **bad) == -1, bad
    for over in (dict(k=0), dict(k=264), dict(r=0), dict(v=0), dict(v=776), dict(k_token=1020), dict(k_token=64), dict(k_head=100),
                 dict(k_head=132), dict(v_head=64), dict(v_token=0), dict(r_token=60), dict(r_token=68), dict(key_start=0),
                 dict(n_keys=-1), dict(dtype=2)):
        assert _prefill(lib, _keys(**over)) == -1, over
    assert _prefill(lib, None) == -1
    assert _prefill(lib, _keys(n_keys=0x7fffffff)) == -2  # 32-bit rows
    assert _prefill(lib, _keys(), Hq=1 << 16) == -2
    assert _prefill(lib, _keys(), n=1 << 28, max_n=1 << 28, max_t=1 << 30) == -2  # 32-bit tile counts
    assert _prefill(lib, _keys(), n=0) == 0 and _prefill(lib, _keys(), max_n=0) == 0
    assert lib.hs2_latent_prefill_workspace(4, 4, 2, 3, 300) > 0
    for bad in ((-1, 4, 2, 3, 300), (4, 0, 2, 3, 300), (4, 4, 0, 3, 300), (4, 4, 2, -3, 300), (4, 4, 2, 3, -1)):
        assert lib.hs2_latent_prefill_workspace(*bad) == 0


def test_binding_refuses_tensors_it_cannot_pass(lib):
    torch = pytest.importorskip("torch")
    bf = torch.bfloat16
    kv = H.KV(k=torch.zeros(4, 1, 64, 576, dtype=bf), v=None, block_table=torch.zeros(2, 2, dtype=torch.int32),
              seq_len=torch.ones(2, dtype=torch.int32))
    rs, rot = torch.zeros(3, dtype=torch.int32), torch.zeros(8, 64)
    c, r, q = torch.zeros(3, 512, dtype=bf), torch.zeros(3, 64, dtype=bf), torch.zeros(3, 4, 64, dtype=bf)
    for bad in (lambda: H.hs2_latent_write(kv, c, r, rs, rot),  # host tensors
                lambda: H.hs2_latent_write(kv, c.float(), r, rs, rot), lambda: H.hs2_latent_write(kv, c[:, :256], r, rs, rot),
                lambda: H.hs2_latent_write(kv, c, r, rs, rot, style="thirds"), lambda: H.hs2_latent_write(kv, c, r, rs, rot.double()),
                lambda: H.hs2_latent_write(kv, c, r, rs, rot, q_out=q), lambda: H.hs2_latent_write(kv, c, r, rs, rot, q=q, q_out=q.float()),
                lambda: H.hs2_latent_read(kv, rs, 3), lambda: H.hs2_latent_read(kv, rs, 3, dtype=torch.float16),
                lambda: H.hs2_latent_chunk(torch.zeros(3, 4, 576, dtype=bf), rs, kv, 0.1, 1),
                lambda: H.hs2_latent_chunk(torch.zeros(3, 4, 576), rs, kv, 0.1, 1),
                lambda: H.hs2_latent_chunk(torch.zeros(3, 4, 512, dtype=bf), rs, kv, 0.1, 1)):
        with pytest.raises(H.HS2Error):
            bad()
    full = H.KV(k=torch.zeros(4, 2, 64, 64, dtype=bf), v=torch.zeros(4, 2, 64, 64, dtype=bf), block_table=kv.block_table,
                seq_len=kv.seq_len)
    rows = torch.zeros(3, 2, 64, dtype=bf)
    for bad in (lambda: H.hs2_latent_read(full, rs, 3), lambda: H.hs2_kv_write_rot(full, rows, rows, rs, rot),
                lambda: H.hs2_kv_write_rot(full, rows, None, rs, rot), lambda: H.hs2_kv_write_rot(full, rows, rows, rs, rot, q=rows.float()),
                lambda: H.hs2_kv_write_rot(full, rows, rows, rs, rot, q_out=rows),
                lambda: H.hs2_kv_write_rot(full, rows, rows, rs, rot, q=rows, q_out=rows.float())):
        with pytest.raises(H.HS2Error):
            bad()
    k = torch.zeros(5, 4, 128, dtype=bf)
    for bad in (lambda: H.hs2_latent_prefill(torch.zeros(3, 4, 192, dtype=bf), k, torch.zeros(5, 64, dtype=bf), k, rs, rs, 0.1, 1, 5),
                lambda: H.hs2_latent_prefill(torch.zeros(3, 4, 192), k, torch.zeros(5, 64, dtype=bf), k, rs, rs, 0.1, 1, 5),
                lambda: H.hs2_latent_prefill(torch.zeros(3, 4, 128, dtype=bf), k, torch.zeros(5, 64, dtype=bf), k, rs, rs, 0.1, 1, 5),
                lambda: H.hs2_latent_prefill(torch.zeros(3, 4, 192, dtype=bf), k, torch.zeros(4, 64, dtype=bf), k, rs, rs, 0.1, 1, 5),
                lambda: H.hs2_latent_prefill(torch.zeros(3, 4, 192, dtype=bf), k, torch.zeros(5, 64, dtype=bf), k, rs, rs[:2], 0.1, 1, 5)):
        with pytest.raises(H.HS2Error):
            bad()
