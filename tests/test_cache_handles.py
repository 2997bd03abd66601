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
