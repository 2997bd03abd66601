"""Table entries that point at free pages, where the page books meet them: flagged, and nothing of
another sequence's comes to be shared."""
import numpy as np
import pytest

import cache_testutil as T
from test_gpu_pages import H, dev  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp4"])
def test_fork_of_a_free_last_page(H, dtype):  # noqa: F811
    """A source whose partly filled page is free: nothing is copied from it, as from one out of
    range; the branch keeps a page of its own, and other branches are whole."""
    import torch

    rng = np.random.default_rng(35)
    c = T.make_cache(rng, dtype, 8, 1, 64)
    pages = H.Pages.make(8)
    dt, dl = dev(np.full((2, 2), -1)), dev([0, 0])
    H.hs2_pages_grow(pages, dt, dl, dev([100, 70]))
    kv = T.device_cache(H, c, np.zeros((2, 2)), [0, 0])
    kv.block_table, kv.seq_len = dt, dl
    dt[0, 1] = 7  # a free page at the far end of the stack
    before = T.cache_arrays(kv, c)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    t, n = H.hs2_pages_fork(pages, [kv], dev([0, 1]), dev_err=err)
    assert int(err.item()) == H.DEV_BAD_PAGE
    assert n.tolist() == [100, 70] and int(pages.ref[7]) == 0
    after = T.cache_arrays(kv, c)
    mine, other, source = int(t[0, 1]), int(t[1, 1]), int(dt[1, 1])
    assert int(pages.ref[mine]) == 1 and int(pages.ref[other]) == 1
    for name in after:
        np.testing.assert_array_equal(after[name][mine], before[name][mine], err_msg=name)
        rows = slice(None) if name.endswith("scale") else (slice(None), slice(0, 6))
        np.testing.assert_array_equal(after[name][other][rows], before[name][source][rows], err_msg=name)


def test_compact_flags_entries_of_free_pages_below(H):  # noqa: F811
    """An entry that points at a free page below the count of referenced ones, which another
    sequence's page moves into: flagged and left as it is."""
    import torch

    rng = np.random.default_rng(36)
    c = T.make_cache(rng, "bf16", 6, 1, 64)
    pages = H.Pages.make(6)
    pages.ref.copy_(dev([0, 1, 0, 0, 1, 0]))
    dt, dl = dev([[4, 1], [0, -1], [1, -1]]), dev([128, 60, 64])
    kv = T.device_cache(H, c, np.zeros((3, 2)), [0, 0, 0])
    kv.block_table, kv.seq_len = dt, dl
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    H.hs2_pages_compact(pages, [kv], dev_err=err)
    assert int(err.item()) == H.DEV_BAD_PAGE
    assert dt.tolist() == [[0, 1], [0, -1], [1, -1]] and pages.ref.tolist() == [1, 1, 0, 0, 0, 0]
    err.zero_()
    dl[1] = 0  # the sequence that pointed there ends: nothing to flag
    H.hs2_pages_compact(pages, [kv], dev_err=err)
    assert int(err.item()) == 0 and dt.tolist() == [[0, 1], [0, -1], [1, -1]]
