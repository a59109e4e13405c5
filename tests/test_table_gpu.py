"""pkv_table_update and the device page pool (GPU) against the plain
allocator of tree_ref: every table entry, the pool, slots and positions are
equal, over sequences of calls that grow, shrink, release and fail."""
import numpy as np
import pytest
import torch

import paged_kv_decode_append_gb300 as pkv

import tree_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"
HEAD = pkv.api.POOL_HEADER


def i32(x):
    return torch.as_tensor(np.ascontiguousarray(x, dtype=np.int32), device=DEV)


class Pair:
    """A device pool with its tables beside the plain one."""

    def __init__(self, num_pages, batch, width, P, seed=None):
        self.pool, self.P = pkv.device_pool(num_pages), P
        ring = None
        if seed is not None:
            ring = np.random.default_rng(seed).permutation(num_pages - 1) + 1
            self.pool[HEAD:] = i32(ring)
        self.plain = ref.TablePool(num_pages, batch, width, P, ring)
        self.table = torch.zeros(batch, width, dtype=torch.int32, device=DEV)
        self.held = torch.zeros(batch, dtype=torch.int32, device=DEV)
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def update(self, lens, new, max_tokens=None, listed=True):
        B = len(lens)
        if max_tokens is None:
            max_tokens = int(sum(max(0, n) for n, L in zip(new, lens) if L >= 0)) + 5
        indptr = torch.full((B + 1,), 9, dtype=torch.int32, device=DEV)
        slots = torch.full((max_tokens,), 9, dtype=torch.int64, device=DEV) if listed else None
        pos = torch.full((max_tokens,), 9, dtype=torch.int32, device=DEV) if listed else None
        self.err.zero_()
        pkv.pkv_table_update(self.pool, self.table, self.held, i32(lens), i32(new), self.P, indptr=indptr,
                             slot_map=slots, positions=pos, err_flag=self.err)
        want = self.plain.update(lens, new, max_tokens if listed else None)
        assert np.array_equal(indptr.cpu().numpy(), want[0])
        if listed:
            assert np.array_equal(slots.cpu().numpy(), want[1])
            assert np.array_equal(pos.cpu().numpy(), want[2])
        assert np.array_equal(self.table.cpu().numpy(), self.plain.table)
        assert np.array_equal(self.held.cpu().numpy(), self.plain.held)
        head, count, ticket = self.pool[:3].tolist()
        ring = self.pool[HEAD:].cpu().numpy()
        assert ticket == 0 and count == len(self.plain.free)
        assert np.array_equal(np.roll(ring, -head)[:count], self.plain.free)
        bits = {"qlen": pkv.api.ERR_QLEN, "overflow": pkv.api.ERR_OVERFLOW, "pool": pkv.api.ERR_POOL}
        assert int(self.err.item()) == int(np.bitwise_or.reduce([0] + [bits[w] for w in want[3].values()]))
        return want


@pytest.mark.parametrize("P", [1, 8, 16, 256])
@pytest.mark.parametrize("B", [1, 3, 64, 257, 1024])
def test_sequences_of_updates(B, P):
    """Rows come, grow by odd counts, shrink (as after rejected drafts), end."""
    rng = np.random.default_rng(B + P)
    top = 40 * P if P < 256 else 3 * P
    width = -(-2 * top // P) + 1
    pair = Pair(B * width // 2 + 8, B, width, P, seed=B)
    lens = np.full(B, -1)
    for _ in range(7):
        fresh = rng.random(B) < 0.5
        lens = np.where(fresh, rng.integers(0, top, B), lens)
        lens = np.where(rng.random(B) < 0.2, -1, lens)
        new = rng.integers(0, 2 * P + 3, B)
        want = pair.update(lens, new)
        kept = np.array([b not in want[3] for b in range(B)])
        # some of the new tokens stay
        lens = np.where(kept & (lens >= 0), lens + rng.integers(0, 1 + np.maximum(0, new)), lens)
        lens = np.where(kept, lens, -1)
    pair.update(np.full(B, -1), np.zeros(B, int), listed=False)
    assert int(pair.pool[1]) == len(pair.plain.free) == B * width // 2 + 7
    assert (pair.table == 0).all()


def test_a_long_prompt():
    pair = Pair(5000, 2, 4200, 16, seed=1)
    pair.update([0, 3], [65000, 1])
    pair.update([65000, 4], [1, 300])
    pair.update([10, -1], [0, 0])


def test_a_fresh_pool_hands_out_ascending_pages_like_the_host_pool():
    host, row = pkv.PagePool(40), np.zeros(8, np.int32)
    host.reserve(row, 16, 0, 100)
    pair = Pair(40, 1, 8, 16)
    pair.update([0], [100])
    assert np.array_equal(pair.table[0].cpu().numpy(), row)


def test_rows_that_fail_keep_their_blocks():
    pair = Pair(12, 4, 6, 16)
    pair.update([0, 0, 0, 0], [33, 10, 0, 40])         # 3 + 1 + 0 + 3 of 11 pages
    pair.update([33, 10, 0, 40], [0, 60, 5, 9])        # row 1 wants 4 more: 4 free; row 2 gets none
    pair.update([33, 10, 0, 40], [-1, 1, 2000, 2])     # negative; past the table
    pair.update([33, 10, 0, 40], [4, 3, 0, 2], max_tokens=6)   # rows 0 fits; 1 passes the list; 3 too
    pair.update([-1, 10, 0, -1], [4, 3, 0, 2])
    pair.update([0, 11, 3, 1], [96, 3, 0, 2])


def test_pages_returned_by_a_call_serve_the_next_one():
    pair = Pair(4, 2, 3, 8)
    pair.update([0, -1], [24, 0])     # all three pages
    pair.update([-1, 0], [0, 8])      # row 0 lets go, row 1 finds none yet
    pair.update([-1, 0], [0, 8])
    assert int(pair.held[1]) == 1


def test_without_lists_and_without_new_tokens():
    pool = pkv.device_pool(10)
    table, held = torch.zeros(2, 4, dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    pkv.pkv_table_update(pool, table, held, i32([17, 16]), None, 16)
    assert table.tolist() == [[1, 2, 0, 0], [3, 0, 0, 0]] and held.tolist() == [2, 1]


def test_tokens_behind_the_last_are_marked():
    pool = pkv.device_pool(10)
    table, held = torch.zeros(1, 4, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    slots, pos = torch.zeros(5000, dtype=torch.int64, device=DEV), torch.zeros(5000, dtype=torch.int32, device=DEV)
    pkv.pkv_table_update(pool, table, held, i32([3]), i32([2]), 16, slot_map=slots, positions=pos)
    assert slots[:3].tolist() == [19, 20, -1] and pos[:3].tolist() == [3, 4, -1]
    assert (slots[2:] == -1).all() and (pos[2:] == -1).all()


def test_broken_state_is_reported():
    def fresh():
        pool = pkv.device_pool(10)
        table, held = torch.zeros(2, 4, dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        return pool, table, held, err

    for word, value in ((0, -1), (0, 9), (1, -2), (1, 10)):
        pool, table, held, err = fresh()
        pool[word] = value
        was = pool.clone()
        indptr = i32([9, 9, 9])
        pkv.pkv_table_update(pool, table, held, i32([3, 3]), i32([2, 2]), 16, indptr=indptr, err_flag=err)
        assert int(err.item()) == pkv.api.ERR_POOL and torch.equal(pool, was) and indptr.tolist() == [0, 0, 0]
        assert (table == 0).all() and (held == 0).all()
    pool, table, held, err = fresh()  # gives back what was never taken
    held[1] = 2
    was = pool.clone()
    pkv.pkv_table_update(pool, table, held, i32([3, -1]), i32([2, 2]), 16, err_flag=err)
    assert int(err.item()) == pkv.api.ERR_POOL and torch.equal(pool, was) and held.tolist() == [0, 2]
    pool, table, held, err = fresh()  # held_blocks past the table
    held[0] = 5
    pkv.pkv_table_update(pool, table, held, i32([3, 3]), i32([2, 2]), 16, err_flag=err)
    assert int(err.item()) == pkv.api.ERR_PAGE and table.tolist() == [[0] * 4, [1, 0, 0, 0]] and held.tolist() == [5, 1]
    pool, table, held, err = fresh()  # a page that cannot be
    pool[HEAD] = 77
    slots = torch.zeros(4, dtype=torch.int64, device=DEV)
    pkv.pkv_table_update(pool, table, held, i32([3, 3]), i32([2, 2]), 16, slot_map=slots, err_flag=err)
    assert int(err.item()) == pkv.api.ERR_PAGE and table[:, 0].tolist() == [0, 2]
    assert slots.tolist() == [-1, -1, 35, 36]


def test_rows_past_the_tokens_that_32_bits_count():
    P, wide = 256, 2 ** 23 + 1
    pool = pkv.device_pool(10)
    table = torch.zeros(2, wide, dtype=torch.int32, device=DEV)
    for L in (2 ** 31 - 3, 2 ** 31 - 1):
        held, err = i32([2 ** 23 - 1, 0]), torch.zeros(1, dtype=torch.int32, device=DEV)
        indptr, was = i32([9, 9, 9]), pool[HEAD:].clone()
        slots, pos = torch.zeros(8, dtype=torch.int64, device=DEV), torch.zeros(8, dtype=torch.int32, device=DEV)
        pool[:2] = i32([0, 9])
        table[1] = 0
        pkv.pkv_table_update(pool, table, held, i32([L, 3]), i32([5, 2]), P, indptr=indptr, slot_map=slots,
                             positions=pos, err_flag=err)
        assert int(err.item()) == pkv.api.ERR_OVERFLOW and indptr.tolist() == [0, 0, 2]
        assert held.tolist() == [2 ** 23 - 1, 1] and not table[0].any() and int(table[1, 0]) == 1
        assert slots.tolist() == [P + 3, P + 4] + [-1] * 6 and pos.tolist() == [3, 4] + [-1] * 6
        assert torch.equal(pool[HEAD:], was)


def test_captured_updates_advance_the_pool():
    pair = Pair(300, 16, 8, 16, seed=3)
    lens, new = i32(np.zeros(16)), i32(np.zeros(16))
    indptr = torch.zeros(17, dtype=torch.int32, device=DEV)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        pkv.pkv_table_update(pair.pool, pair.table, pair.held, lens, new, 16, indptr=indptr)
    rng = np.random.default_rng(0)
    for _ in range(5):
        a, b = rng.integers(-1, 90, 16), rng.integers(0, 30, 16)
        lens.copy_(i32(a)), new.copy_(i32(b))
        graph.replay()
        want = pair.plain.update(a, b)
        assert np.array_equal(indptr.cpu().numpy(), want[0])
        assert np.array_equal(pair.table.cpu().numpy(), pair.plain.table)
