"""pt_cache_tables at the ends of its ranges, against counts made by hand."""
import numpy as np
import pytest
import torch

import prefix_tree_block_gb300 as pt

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _built():
    from prefix_tree_block_gb300 import build as b

    b.build()


@pytest.mark.parametrize("small", [0, 2, 15, 31])
def test_rows_that_ask_for_more_than_2_31_tokens(small):
    """The tokens up to max_new get their own rows' slots all the same."""
    n, ps, width, cap, new = 40, 1 << 16, 1 << 12, 3 * (1 << 12), 5000
    added = np.full(n, 1 << 28, np.int64)
    added[:small] = 1000 // max(small, 1) + np.arange(small)
    ring = np.random.default_rng(small).permutation(1 << 20)[:cap].astype(np.int32)
    cuda = lambda x, t=torch.int32: torch.from_numpy(np.ascontiguousarray(x)).to("cuda", t)  # noqa: E731
    tables = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    lens, ctr, row_ptr, slots, pos = pt.cache_tables(
        cuda(np.zeros(n)), cuda(added), tables, cuda(ring), torch.tensor([0, cap], device="cuda"), ps, new, start=cuda(np.arange(n) * 10))
    with pytest.raises(pt.PTError):  # too many tokens for max_new and too few pages
        pt.sync_status()
    pages = -(-added // ps)
    taken = np.minimum(np.cumsum(pages), cap)
    got = np.diff(np.concatenate([[0], taken]))
    first = np.cumsum(added) - added
    np.testing.assert_array_equal(row_ptr.cpu().numpy(), np.minimum(np.cumsum(np.concatenate([[0], added])), (1 << 30) + 1))
    np.testing.assert_array_equal(lens.cpu().numpy(), np.minimum(added, got * ps))
    assert ctr.tolist() == [cap, cap]
    y = np.arange(new)
    row = np.searchsorted(first, y, side="right") - 1
    tok = y - first[row]
    np.testing.assert_array_equal(slots.cpu().numpy(), ring[(taken - got)[row] + tok // ps].astype(np.int64) * ps + tok % ps)
    np.testing.assert_array_equal(pos.cpu().numpy(), row * 10 + tok)
    want = np.full((n, width), -1, np.int32)
    for i in range(n):
        want[i, :got[i]] = ring[taken[i] - got[i]:taken[i]]
    np.testing.assert_array_equal(tables.cpu().numpy(), want)
    pt.sync_status()
