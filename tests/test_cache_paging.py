"""kv_cache_extend, kv_cache_slots and kv_cache_truncate on the GPU against the oracle's integers:
request counts around the block's threads, page sizes that are no powers of two, free lists that run
out, rows and tokens without room, lengths and lists updated in place, and pages that come back."""
import numpy as np
import pytest
import torch

import oracle
from rope_attention_gb300 import native

pytestmark = pytest.mark.gpu


def dev(x, dtype=torch.int32):
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


class Pages:
    def __init__(self, seed, lens, stride, bs, spare, lost=0):
        rng = np.random.default_rng(seed)
        held = [-(-n // bs) for n in lens]
        self.block_num = sum(held) + spare + lost
        ids = rng.permutation(self.block_num).astype(np.int32)
        self.table = np.full((len(lens), stride), -9, np.int32)
        at = 0
        for b, n in enumerate(held):
            self.table[b, :n] = ids[at:at + n]
            at += n
        self.free = np.full(self.block_num, -3, np.int32)
        self.free[:spare] = ids[at:at + spare]
        self.count, self.lens, self.bs = spare, np.array(lens, np.int32), bs

    def params(self, max_tokens=1):
        return native.KvCachePagingParams(B=len(self.lens), block_num=self.block_num, block_size=self.bs,
                                          block_table_stride=self.table.shape[1], max_tokens=max_tokens)

    def extend(self, new, max_tokens, in_place=False):
        """The call and the oracle, which must agree in everything."""
        want = oracle.paging.extend(new, self.lens, self.table, self.free, self.count, block_num=self.block_num,
                                    block_size=self.bs, max_tokens=max_tokens)
        lens, count, table, free = dev(self.lens), dev([self.count]), dev(self.table), dev(self.free)
        index = torch.full((max_tokens + 2,), 77, dtype=torch.int64, device="cuda")
        cu = torch.full((len(self.lens) + 2,), 77, dtype=torch.int32, device="cuda")
        new_lens, new_count = (lens, count) if in_place else (torch.full_like(lens, 77), torch.full_like(count, 77))
        err = dev([5])
        native.kv_cache_extend(self.params(max_tokens), dev(new), lens, table, free, count, index[:max_tokens], cu[:-1], new_lens,
                               new_count, err)
        got = {"index": index[:-2], "cu_seqlens": cu[:-1], "new_seq_lens": new_lens, "table": table}
        for k, t in got.items():
            assert np.array_equal(t.cpu().numpy(), want[k]), (k, np.nonzero(t.cpu().numpy() != want[k]))
        assert int(new_count) == want["new_free_count"] and int(err) == 5 + want["errors"]
        assert (index[-2:] == 77).all() and int(cu[-1]) == 77 and np.array_equal(free.cpu().numpy(), self.free)
        if not in_place:
            assert np.array_equal(lens.cpu().numpy(), self.lens) and int(count) == self.count
        self.table, self.lens, self.count = want["table"], want["new_seq_lens"], want["new_free_count"]
        return want

    def truncate(self, keep, in_place=False):
        want = oracle.paging.truncate(keep, self.lens, self.table, self.free, self.count, block_num=self.block_num, block_size=self.bs)
        lens, count, table, free = dev(self.lens), dev([self.count]), dev(self.table), dev(self.free)
        new_lens, new_count = (lens, count) if in_place else (torch.full_like(lens, 77), torch.full_like(count, 77))
        err = dev([5])
        native.kv_cache_truncate(self.params(), lens, table, free, count, new_lens, new_count,
                                 keep=None if keep is None else dev(keep), dev_error_count=err)
        assert np.array_equal(new_lens.cpu().numpy(), want["new_seq_lens"])
        assert np.array_equal(free.cpu().numpy(), want["free_pages"])
        assert int(new_count) == want["new_free_count"] and int(err) == 5 + want["errors"]
        assert np.array_equal(table.cpu().numpy(), self.table)
        self.lens, self.free, self.count = want["new_seq_lens"], want["free_pages"], want["new_free_count"]
        return want


@pytest.mark.parametrize("B", [1, 2, 31, 33, 256, 1023, 1024, 1025, 3000, 16384])
@pytest.mark.parametrize("bs", [16, 48])
def test_request_counts(B, bs):
    rng = np.random.default_rng(B)
    p = Pages(B, rng.integers(0, 100, B), 12, bs, 2 * B + 3)
    p.extend(rng.integers(-2, 4, B), 4 * B)
    p.truncate(rng.integers(-5, 100, B))


@pytest.mark.parametrize("bs", [1, 2, 16, 32, 96, 128, 1000])
@pytest.mark.parametrize("in_place", [False, True])
def test_page_sizes(bs, in_place):
    rng = np.random.default_rng(bs)
    lens = [0, 1, bs - 1, bs, bs + 1, 3 * bs, 777]
    new = [1, bs, 1, 1, 2 * bs, 0, 500]
    p = Pages(2, lens, 2000 // bs + 7, bs, 4000 // bs + 9)
    p.extend(new, sum(new) + 3, in_place)
    p.extend([0] * 7, 1, in_place)
    p.truncate([0, 1, 0, bs, 2, 3 * bs, 500], in_place)
    p.truncate(None, in_place)
    assert p.count == p.block_num and sorted(p.free) == list(range(p.block_num))


@pytest.mark.parametrize("tokens", [2047, 2048, 2049, 5000, 9000, 20000, 65430, 70000, 400000])
def test_long_prompts(tokens):
    p = Pages(3, [100, 0, 33], tokens // 16 + 20, 16, tokens // 16 + 40)
    p.extend([tokens // 3, tokens - tokens // 3 - 1, 1], tokens + 100)
    p.truncate([50, 0, 34])


def test_long_prompts_in_place_and_refused():
    p = Pages(15, [100, 0, 33, 7], 5000, 16, 6000)
    # 1875 and 3750 pages of 6000; the third's 1250 are not there, the last needs none
    want = p.extend([30000, 60000, 20000, 3], 150000, in_place=True)
    assert want["new_seq_lens"].tolist() == [30100, 60000, 33, 10] and want["errors"] == 1
    p.extend([1, 1, 1, 1], 100000, in_place=True)


@pytest.mark.parametrize("B", [3, 16384])
def test_slots_of_long_contexts(B):
    lens = [300000, 0, 77] if B == 3 else [20] * B
    p = Pages(16, lens, max(lens) // 16 + 2, 16, 3)
    total = sum(lens)
    want = oracle.paging.slots(None, lens, p.table, block_num=p.block_num, block_size=16, max_tokens=total)
    index, cu = torch.empty(total, dtype=torch.int64, device="cuda"), torch.empty(B + 1, dtype=torch.int32, device="cuda")
    native.kv_cache_slots(p.params(total), dev(lens), dev(p.table), index, cu)
    assert np.array_equal(index.cpu().numpy(), want["index"]) and np.array_equal(cu.cpu().numpy(), want["cu_seqlens"])


def test_free_list_that_runs_out():
    # 7 pages: the third request is refused, and whoever needs pages behind it; the last needs none
    p = Pages(4, [30, 32, 0, 5, 31, 1], 10, 16, 7)
    want = p.extend([40, 40, 60, 20, 1, 10], 200)
    assert want["new_seq_lens"].tolist() == [70, 72, 0, 5, 32, 11] and want["errors"] == 2 and want["new_free_count"] == 1
    p.extend([1, 1, 1, 1, 1, 1], 200)
    p = Pages(5, [3, 4], 5, 16, 0)
    p.extend([10, 20], 30)


def test_rows_and_tokens_without_room():
    p = Pages(6, [60, 10, 10, 10], 4, 16, 20)
    want = p.extend([5, 5, 60, 3], 70)     # the first passes its row; the last passes max_tokens
    assert want["new_seq_lens"].tolist() == [60, 15, 10, 10] and want["errors"] == 3
    p.extend([2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, 1], 50)
    p.extend([0, 0, 0, 1], 1)


def test_lengths_counts_and_pages_out_of_range():
    p = Pages(7, [40, 20], 4, 16, 5)
    p.lens = np.array([-7, 1000], np.int32)
    p.extend([3, 3], 10)
    p = Pages(8, [40, 20], 8, 16, 5)
    p.table[0, 2] = 1 << 20                # the page that the first new tokens are in
    want = p.extend([10, 10], 20)
    assert want["errors"] == 8
    p = Pages(9, [40, 40], 8, 16, 5)
    p.table[1, 0] = -1
    p.truncate([0, 0])
    p = Pages(10, [40, 40], 8, 16, 5)
    p.count = p.block_num - 2              # a list that says it has more than it can
    p.truncate([0, 16])
    p = Pages(11, [40, 40], 8, 16, 5)
    p.count = 1000
    p.truncate([0, 16])
    p.count = -4
    p.extend([1, 100], 101)


@pytest.mark.parametrize("B,bs", [(1, 16), (32, 128), (1500, 48)])
@pytest.mark.parametrize("with_starts", [False, True])
def test_slots(B, bs, with_starts):
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 300, B)
    p = Pages(12, lens, 300 // bs + 2, bs, 3)
    starts = rng.integers(-3, 40, B) if with_starts else None
    counts = rng.integers(-2, 300, B)      # some reach behind their pages and rows
    total = int(np.maximum(counts, 0).sum())
    for room in (total + 9, max(1, total - 50)):
        want = oracle.paging.slots(starts, counts, p.table, block_num=p.block_num, block_size=bs, max_tokens=room)
        index = torch.full((room + 1,), 77, dtype=torch.int64, device="cuda")
        cu, err = torch.empty(B + 1, dtype=torch.int32, device="cuda"), dev([0])
        native.kv_cache_slots(p.params(room), dev(counts), dev(p.table), index[:room], cu,
                              starts=None if starts is None else dev(starts), dev_error_count=err)
        assert np.array_equal(index[:-1].cpu().numpy(), want["index"]) and int(index[-1]) == 77
        assert np.array_equal(cu.cpu().numpy(), want["cu_seqlens"]) and int(err) == want["errors"]


def test_truncate_undoes_extend():
    rng = np.random.default_rng(0)
    p = Pages(13, rng.integers(0, 200, 50), 40, 16, 600)
    free, lens = p.free.copy(), p.lens.copy()
    p.extend(rng.integers(0, 150, 50), 8000)
    p.truncate(lens)
    assert np.array_equal(p.free, free) and np.array_equal(p.lens, lens)


def test_a_graph_of_steps_in_place():
    """A captured step extends every request by one token; replayed, it goes on from its own state."""
    rng = np.random.default_rng(1)
    p = Pages(14, rng.integers(0, 60, 40), 12, 16, 200)
    B, T = 40, 48
    lens, count, table, free = dev(p.lens), dev([p.count]), dev(p.table), dev(p.free)
    index, cu, new, err = torch.empty(T, dtype=torch.int64, device="cuda"), torch.empty(B + 1, dtype=torch.int32, device="cuda"), dev([1] * B), dev([0])
    step = lambda: native.kv_cache_extend(p.params(T), new, lens, table, free, count, index, cu, lens, count, err)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        step()
    side = torch.cuda.Stream()
    for _ in range(40):
        want = oracle.paging.extend([1] * B, p.lens, p.table, p.free, p.count, block_num=p.block_num, block_size=16, max_tokens=T)
        with torch.cuda.stream(side):
            g.replay()
        side.synchronize()
        assert np.array_equal(index.cpu().numpy(), want["index"]) and np.array_equal(lens.cpu().numpy(), want["new_seq_lens"])
        assert np.array_equal(table.cpu().numpy(), want["table"]) and int(count) == want["new_free_count"]
        p.lens, p.table, p.count = want["new_seq_lens"], want["table"], want["new_free_count"]
    assert int(err) == 0
