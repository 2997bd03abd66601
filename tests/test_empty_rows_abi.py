"""Calls without rows do nothing, whether or not they name queries: an empty tensor has no address."""
import ctypes

import pytest

from top_hs2_fa_gb300 import build
from top_hs2_fa_gb300 import hs2 as H


@pytest.fixture(scope="module")
def lib():
    build.build()
    return H.load()


def _kv(**over):
    return H.hs2_kv(**{**dict(k=16, v=32, block_table=48, seq_len=64, batch=2, num_pages=10, max_pages=5, page_size=64, Hkv=2,
                              d=128, dtype=1), **over})


ROT = H.hs2_rot(table=16, n_pos=100, dim=64, pairs=0)


def _write_rot(lib, n=0, k=0, v=0, q=0, Hq=4, qo=0, rs=1024):
    return lib.hs2_kv_write_rot(ctypes.byref(_kv()), k, 256, v, 256, 1, rs, n, ctypes.byref(ROT), q, 512, Hq, qo, 512, None, None)


def _latent_write(lib, n=0, c=0, r=0, q=0, Hq=16, qo=0, rs=1024):
    return lib.hs2_latent_write(ctypes.byref(_kv(v=0, Hkv=1, d=576)), c, 512, r, 64, 1, rs, n, ctypes.byref(ROT), q, 16 * 64, 64, Hq,
                                qo, 16 * 576, 576, None, None)


@pytest.mark.parametrize("call", [_write_rot, _latent_write])
def test_no_rows_with_queries(lib, call):
    for args in (dict(), dict(Hq=0), dict(q=2048), dict(qo=4096), dict(q=2048, qo=4096)):
        assert call(lib, **args) == 0, args
    for args in (dict(Hq=-1), dict(rs=0), dict(n=-1)):  # (refused as with rows)
        assert call(lib, **args) == -1, args
    rows = dict(n=3, **({"k": 256, "v": 512} if call is _write_rot else {"c": 256, "r": 1280}))
    for args in (dict(), dict(q=2048), dict(qo=4096), dict(q=2048, qo=4096, Hq=0)):  # with rows, queries go with q_out
        assert call(lib, **rows, **args) == -1, args
