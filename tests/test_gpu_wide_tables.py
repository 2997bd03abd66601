"""Tables of more positions than 32 bits count."""
import numpy as np
import pytest

import cache_testutil as T
from test_gpu_chunk import H  # noqa: F401
from test_gpu_row_starts import flags

pytestmark = pytest.mark.gpu


def test_tables_beyond_32_bits_of_positions(H):  # noqa: F811
    """A table of 2^25 columns (2^31 positions): lengths within it are lengths."""
    import torch

    rng = np.random.default_rng(94)
    c = T.make_cache(rng, "bf16", 4, 1, 64)
    table = torch.full((1, 1 << 25), -1, dtype=torch.int32, device="cuda")
    table[0, :2] = torch.tensor([3, 1], dtype=torch.int32)
    small = T.device_cache(H, c, np.array([[3, 1]]), [100])
    wide = H.KV(k=small.k.clone(), v=small.v.clone(), block_table=table, seq_len=small.seq_len)
    rows = torch.tensor(rng.standard_normal((90, 1, 64)), dtype=torch.bfloat16, device="cuda")
    drs = T.device(np.array([0, 90], np.int32))
    for kv in (small, wide):
        assert flags(H, lambda e: H.hs2_kv_write(kv, rows, rows, drs, dev_err=e)) == 0
    assert torch.equal(small.k, wide.k) and torch.equal(small.v, wide.v)
    got = [H.hs2_kv_read(kv, drs, 90) for kv in (small, wide)]
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][0][:, 0], rows[:, 0].float())
