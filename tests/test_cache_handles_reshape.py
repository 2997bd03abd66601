"""Handles whose tensors change in place without a change of address or size."""
import pytest

torch = pytest.importorskip("torch")

from top_hs2_fa_gb300 import hs2 as H  # noqa: E402
from test_cache_handles import kv  # noqa: E402


def test_a_table_reshaped_in_place_is_seen():
    a = kv()
    assert a._cached()[0].max_pages == 2
    a.block_table.resize_(2, 3)
    assert a._cached()[0].max_pages == 3
    a.block_table.resize_(6, 1)
    assert a._cached()[0].max_pages == 1


def test_a_pool_reshaped_in_place_is_seen():
    a = kv()
    assert (a._cached()[0].num_pages, a._cached()[0].Hkv, a._cached()[0].d) == (4, 2, 64)
    a.k.data = a.k.data.view(8, 1, 64, 64)
    assert (a._cached()[0].num_pages, a._cached()[0].Hkv) == (8, 1)
    a.k.data = a.k.data.view(4, 1, 64, 128)
    assert (a._cached()[0].num_pages, a._cached()[0].d) == (4, 128)


def test_a_pool_of_another_type_is_seen():
    a = kv()
    a._cached()
    a.k.data = a.k.data.view(torch.float16)  # the same bytes, not a cache's type
    with pytest.raises(H.HS2Error):
        a._cached()


@pytest.mark.parametrize("name", ["k", "v", "block_table"])
def test_a_tensor_transposed_in_place_is_refused(name):
    a = kv()
    if name == "block_table":
        a.block_table = torch.zeros(3, 3, dtype=torch.int32)
    a._cached()
    t = getattr(a, name)
    t.transpose_(0, 1)  # a square table keeps its shape
    with pytest.raises(H.HS2Error):
        a._cached()


def test_books_that_change_shape_in_place_are_refused():
    p = H.Pages.make(6, "cpu")
    p._cached()
    p.ref.resize_(2, 3)
    with pytest.raises(H.HS2Error):
        p._cached()
    p = H.Pages.make(6, "cpu")
    p._cached()
    p.free_list.data = p.free_list.data.view(torch.float32)
    with pytest.raises(H.HS2Error):
        p._cached()
