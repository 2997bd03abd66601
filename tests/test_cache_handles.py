"""Handles of caches and page pools: copies, and tensors that change under them."""
import copy
import pickle

import pytest

torch = pytest.importorskip("torch")

from top_hs2_fa_gb300 import hs2 as H  # noqa: E402


def kv():
    return H.KV(k=torch.zeros(4, 2, 64, 64, dtype=torch.bfloat16), v=torch.zeros(4, 2, 64, 64, dtype=torch.bfloat16),
                block_table=torch.zeros(3, 2, dtype=torch.int32), seq_len=torch.ones(3, dtype=torch.int32))


@pytest.mark.parametrize("make", [kv, lambda: H.Pages.make(5, "cpu")])
def test_used_handles_are_copied_and_pickled(make):
    a = make()
    a._cached()
    for b in (copy.copy(a), copy.deepcopy(a), pickle.loads(pickle.dumps(a))):
        got = b._cached()
        assert got[3] == tuple(t.data_ptr() for t in b._tensors())
        assert b.c().num_pages == a.c().num_pages


def test_changed_tensors_are_seen():
    a = kv()
    first = a._cached()
    assert a._cached() is first
    a.seq_len = torch.ones(2, dtype=torch.int32)
    assert a._cached()[0].batch == 2
    a.block_table.resize_(3, 1)  # in place, at the same address
    assert a._cached()[0].max_pages == 1
    a.k.data = torch.zeros(6, 2, 64, 64, dtype=torch.bfloat16)
    assert a._cached()[0].num_pages == 6 and a._cached()[0].k == a.k.data_ptr()
    a.c().batch = 77  # a caller's own struct
    assert a._cached()[0].batch == 2


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8", "fp4"])
def test_a_chunk_workspace_suffices_for_smaller_calls(dtype):
    import ctypes
    import random

    from top_hs2_fa_gb300 import build
    build.build()
    lib, rng = H.load(), random.Random(7)
    code = {"f32": H.F32, "bf16": H.BF16, "fp8": H.FP8_E4M3, "fp4": H.FP4_E2M1}[dtype]
    size = lambda: int(2 ** rng.uniform(0, 17))  # noqa: E731
    for _ in range(3000):
        Hkv, G = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 4, 8, 16, 32))
        c = H.hs2_kv(batch=rng.choice((1, 3, 17, 200)), num_pages=1000, max_pages=1 << 12, page_size=64, Hkv=Hkv,
                     d=rng.choice((64, 128)), dtype=code)
        w = rng.choice((0, 0, size()))
        big = [size(), size(), size()]
        small = [max(1, int(x * rng.choice((1, 1, 0.9, 0.5, rng.random())))) for x in big]
        need = [lib.hs2_fa_chunk_workspace(n, Hkv * G, ctypes.byref(c), max_n, max_t, w) for n, max_n, max_t in (big, small)]
        assert need[1] <= need[0], (big, small, w, Hkv, G, c.batch, c.d, need)
