"""A pool of the most pages that cp_spec_kv_plan allows: counts next to 2^31."""
import pytest

import kv16_reference as R
from gpu_common import require_gpu, torch

pytestmark = pytest.mark.gpu


def test_all_pages_of_the_largest_pool():
    """16 sequences take 2^31 - 16 pages in one step and give them back in the next."""
    require_gpu()
    from speculative_decoding_rvq_gb300 import binding as b
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    n_pages, n, page = (1 << 31) - 1, 16, 16
    most = n_pages // n
    pool = b.PagePool(n_pages, page, n, most)
    rows = pool.plan(R.ints([most * page] * n))
    assert rows.refused.tolist() == [0] * n and rows.kv_len.tolist() == [most * page] * n
    assert pool.held.tolist() == [most] * n and pool.n_free.item() == n_pages - n * most
    for i in range(n):  # the top of the stack was page 0
        assert torch.equal(pool.pages[i], torch.arange(i * most, (i + 1) * most, dtype=torch.int32, device="cuda")), i
    rows = pool.plan(R.ints([0] * n))
    assert rows.kv_len.tolist() == [0] * n and pool.n_free.item() == n_pages and pool.held.tolist() == [0] * n
    for i in range(n):
        assert (pool.pages[i] == -1).all(), i
        lo, hi = i * most, (i + 1) * most
        assert torch.equal(pool.free[lo: hi], torch.arange(n_pages - 1 - lo, n_pages - 1 - hi, -1, dtype=torch.int32, device="cuda")), i
    del pool
    torch.cuda.empty_cache()
