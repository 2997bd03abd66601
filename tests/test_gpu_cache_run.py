"""A run of the paged-cache operators over quantised caches with every attention compared with the 64-bit
form on the codes that the run itself wrote, and those codes with exact quantisation. Tolerances as
in the tests of hs2_fa_chunk."""
import numpy as np
import pytest

import cache_testutil as T
from test_gpu_chunk import H, check  # noqa: F401
from test_gpu_pages import dev

pytestmark = pytest.mark.gpu


def of_device(kv, c):
    return dict(c, **T.cache_arrays(kv, c))


@pytest.mark.parametrize("dtype", ["fp8", "fp4"])
@pytest.mark.parametrize("d,Hkv", [(64, 2), (128, 1)])
def test_run_against_64_bits(H, dtype, d, Hkv):  # noqa: F811
    """Prompts admitted, written and attended; branches forked, grown by a draft token each and
    verified; the pool compacted, and the branches attend again."""
    import torch

    rng = np.random.default_rng(42)
    NP, Hq, W = 64, 8, 12
    counts, src = [70, 1, 64, 430], [3, 3, 0, -1, 1]
    c = T.make_cache(rng, dtype, NP, Hkv, d, scale=1.0)
    pages = H.Pages.make(NP)
    kv = T.device_cache(H, c, np.full((4, W), -1), np.zeros(4))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def rows(n):
        raw = [T.bf16_round(rng.standard_normal((n, h, d)).astype(np.float32)) for h in (Hkv, Hkv, Hq)]
        return [T.device(x) for x in raw], [T.widen(x) for x in raw]

    def write_and_attend(cache, new, first):
        """New rows in, compared bit for bit; attention over them, compared with 64 bits."""
        lens, bt = T.host(cache.seq_len).tolist(), T.host(cache.block_table)
        (k, v, q), (kx, vx, qx) = rows(sum(new))
        rs = T.starts(new)
        before = of_device(cache, c)
        H.hs2_kv_write(cache, k, v, dev(rs), dev_err=err)
        r, pg, ln = T.places(rs, [t if n else 0 for t, n in zip(lens, new)], bt)
        want = T.write_rows(T.write_rows(before, kx, "k", r, pg, ln), vx, "v", r, pg, ln)
        now = of_device(cache, c)
        for name in T.cache_arrays(cache, c):
            np.testing.assert_array_equal(now[name], want[name], err_msg=name)
        o, lse = H.hs2_fa_chunk(q, dev(rs), cache, d ** -0.5, max(new), max_t=max(lens), dev_err=err)
        check((o.double().cpu().numpy(), lse.cpu().numpy()), T.attend(now, qx, rs, lens, bt, d ** -0.5), dtype)
        return q, qx, rs, o, lse

    H.hs2_pages_grow(pages, kv.block_table, kv.seq_len, dev(counts), dev_err=err)
    write_and_attend(kv, counts, True)
    ct, cl = H.hs2_pages_fork(pages, [kv], dev(src), dev_err=err)
    one = [int(s >= 0) for s in src]
    H.hs2_pages_grow(pages, ct, cl, dev(one), dev_err=err)
    child = H.KV(k=kv.k, v=kv.v, block_table=ct, seq_len=cl, k_scale=kv.k_scale, v_scale=kv.v_scale, k_sf=kv.k_sf,
                 v_sf=kv.v_sf)
    q, qx, rs, o, lse = write_and_attend(child, one, False)
    # the first prompt ends, the rest moves to the pool's front
    H.hs2_pages_free(pages, kv.block_table, kv.seq_len, dev([1, 0, 0, 0]), dev_err=err)
    kv.seq_len[0] = 0
    both = H.KV(k=kv.k, v=kv.v, block_table=torch.cat((kv.block_table, ct)), seq_len=torch.cat((kv.seq_len, cl)),
                k_scale=kv.k_scale, v_scale=kv.v_scale, k_sf=kv.k_sf, v_sf=kv.v_sf)
    H.hs2_pages_compact(pages, [both], dev_err=err)
    live = NP - int(pages.n_free)
    child.block_table = both.block_table[4:].contiguous()
    assert all(int(child.block_table[b, 0]) < live for b, n in enumerate(one) if n)
    o2, lse2 = H.hs2_fa_chunk(q, dev(rs), child, d ** -0.5, 1, max_t=W * 64, dev_err=err)
    want = T.attend(of_device(child, c), qx, rs, T.host(cl).tolist(), T.host(child.block_table), d ** -0.5)
    check((o2.double().cpu().numpy(), lse2.cpu().numpy()), want, dtype)
    kv.block_table = both.block_table[:4].contiguous()
    H.hs2_pages_free(pages, kv.block_table, kv.seq_len, dev([1] * 4), dev_err=err)
    H.hs2_pages_free(pages, child.block_table, cl, dev([1] * 5), dev_err=err)
    assert int(err.item()) == 0 and int(pages.n_free) == NP and (pages.ref == 0).all()
