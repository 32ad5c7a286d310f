"""The paging calls at the ends of what they document, on the GPU: positions around 2^31 - 256, and
requests that gave pages away before they end."""
import numpy as np
import pytest
import torch

from rope_attention_gb300 import native
from test_cache_paging import Pages, dev

pytestmark = pytest.mark.gpu

END = 2 ** 31 - 256                    # positions of a row are below this


def test_positions_at_the_end_of_31_bits():
    # one row of 128 pages of 2^24 slots: 2^31 positions, of which the last 256 are none
    bs, stride = 1 << 24, 128
    p = native.KvCachePagingParams(B=1, block_num=200, block_size=bs, block_table_stride=stride, max_tokens=12)
    table = torch.arange(stride - 1, -1, -1, dtype=torch.int32, device="cuda").view(1, stride)   # the last page is page 0
    index, cu, err = torch.empty(12, dtype=torch.int64, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda"), dev([0])
    native.kv_cache_slots(p, dev([8]), table, index, cu, starts=dev([END - 3]), dev_error_count=err)
    first = END - 3 - (stride - 1) * bs
    assert index.tolist() == [first, first + 1, first + 2] + [-1] * 9 and cu.tolist() == [0, 8] and int(err) == 5
    native.kv_cache_slots(p, dev([2]), table, index, cu, starts=dev([2 ** 31 - 1]), dev_error_count=err)
    assert index.tolist() == [-1] * 12 and int(err) == 7
    # a request just short of the end: as much as fits, and no more
    free, count = torch.full((200,), 150, dtype=torch.int32, device="cuda"), dev([3])
    for new, lens, want, errors in ((3, END - 3, END, 0), (4, END - 3, END - 3, 1), (1, 2 ** 31 - 1, END, 1), (0, 2 ** 31 - 1, END, 0)):
        err.zero_()
        got, left = dev([0]), dev([0])
        native.kv_cache_extend(p, dev([new]), dev([lens]), table, free, count, index, cu, got, left, err)
        assert int(got) == want and int(left) == 3 and int(err) == errors, (new, lens)
        assert index.tolist() == ([first, first + 1, first + 2] + [-1] * 9 if want == END and new == 3 else [-1] * 12)
    # cut back to the first page: the other 127 come back
    err.zero_()
    got, left = dev([0]), dev([0])
    native.kv_cache_truncate(p, dev([2 ** 31 - 1]), table, free, count, got, left, keep=dev([1]), dev_error_count=err)
    assert int(got) == 1 and int(left) == 130 and int(err) == 0
    assert free[3:130].tolist() == list(range(127))


@pytest.mark.parametrize("away", [0, 1, 5])
def test_requests_that_gave_pages_away_end(away):
    """The first `away` pages of each request went to another one, and their entries are -1."""
    rng = np.random.default_rng(away)
    p = Pages(17, rng.integers(16 * away + 1, 300, 40), 20, 16, 30)
    gone = p.table[:, :away].copy()
    p.table[:, :away] = -1
    given = list(p.free[:p.count])
    want = p.truncate(None)
    assert want["errors"] == 40 * away and p.count == p.block_num - 40 * away
    back = p.free[:p.count].tolist()
    assert len(set(back)) == len(back) and not set(back) & set(gone.ravel().tolist()) and back[:30] == given
