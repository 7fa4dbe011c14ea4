"""The page bookkeeping of a sequence that has been sliding for long: what it keeps and does depends
on the pages that the sequence has, not on how many it ever had."""
import time

import numpy as np
import pytest

from block_causal_attention_b200 import PagePool
from block_causal_attention_b200.streaming import PagedWindow

PAGE = 128


class ListPool:
    """What PagePool says of its rows, with a plain list of pages a sequence."""

    def __init__(self, pages):
        self.users, self.rows = [0] * pages, {}

    def take(self):
        p = self.users.index(0)
        self.users[p] = 1
        return p

    def grow(self, s, begin, end):
        row, moves = self.rows[s], []
        if begin == end:
            return moves
        first, last = begin // PAGE, -(-end // PAGE)
        shared = [i for i in range(first, min(last, len(row))) if row[i] < 0 or self.users[row[i]] > 1]
        if len(shared) + max(0, last - max(first, len(row))) > self.users.count(0):
            raise MemoryError
        for i in shared:
            old, row[i] = row[i], self.take()
            if old >= 0:
                self.users[old] -= 1
                if i * PAGE < begin or (i + 1) * PAGE > end:
                    moves.append((old, row[i]))
        while len(row) < last:
            row.append(self.take() if len(row) >= first else -1)
        return moves

    def release(self, s, token):
        row = self.rows[s]
        for i in range(min(max(token, 0) // PAGE, len(row))):
            if row[i] >= 0:
                self.users[row[i]] -= 1
            row[i] = -1

    def fork(self, s, new):
        self.rows[new] = list(self.rows[s])
        for p in self.rows[s]:
            if p >= 0:
                self.users[p] += 1

    def close(self, s):
        self.release(s, len(self.rows[s]) * PAGE)
        del self.rows[s]


@pytest.mark.parametrize("seed", range(6))
def test_rows_moves_and_tables_as_with_plain_lists(seed):
    """Any order of growing (ahead of the end, in released pages, with gaps), releasing, forking,
    closing and compacting: the same pages, copies, tables and refusals."""
    rng = np.random.default_rng(seed)
    pool, want = PagePool(30), ListPool(30)
    for _ in range(1500):
        op = rng.integers(0, 12)
        s = int(rng.choice(list(want.rows))) if want.rows else None
        if s is None or (op == 0 and len(want.rows) < 6):
            want.rows[pool.open()] = []
        elif op <= 5:
            n = len(want.rows[s]) * PAGE
            begin = int(rng.integers(0, n + 600)) if op < 3 else max(0, n - int(rng.integers(0, 300)))
            end = begin + int(rng.integers(0, 700))
            try:
                moves = want.grow(s, begin, end)
            except MemoryError:
                with pytest.raises(MemoryError):
                    pool.grow(s, begin, end)
                want.close(s)
                pool.close(s)
            else:
                assert pool.grow(s, begin, end) == moves
        elif op <= 8:
            token = int(rng.integers(-50, len(want.rows[s]) * PAGE + 400))
            want.release(s, token)
            pool.release_before(s, token)
        elif op == 9 and len(want.rows) < 6:
            want.fork(s, pool.fork(s))
        elif op == 10:
            want.close(s)
            pool.close(s)
        else:
            used = sum(u > 0 for u in want.users)
            high = [p for p in range(used, 30) if want.users[p]]
            moves = list(zip(high, [p for p in range(used) if not want.users[p]]))
            assert pool.compact() == moves
            for a, b in moves:
                want.users[a], want.users[b] = 0, want.users[a]
                want.rows = {k: [b if p == a else p for p in row] for k, row in want.rows.items()}
        assert pool.free_pages == want.users.count(0)
        for k, row in want.rows.items():
            assert pool.row(k) == row
            at = int(rng.integers(0, len(row) + 3))
            assert pool.row(k, at) == row[at:]
        order = [int(k) for k in rng.permutation(list(want.rows))]
        width = max((len(want.rows[k]) for k in order), default=0)
        table = pool.table(order)
        assert table.shape == (len(order), width) and table.dtype == np.int32
        assert [t[:len(want.rows[k])].tolist() for t, k in zip(table, order)] == [want.rows[k] for k in order]


def test_a_sequence_far_on_keeps_only_its_pages():
    """Absolute token 10^12: a list entry a page passed over would be 8 * 10^9 of them."""
    p = PagePool(8)
    a = p.open()
    far = 10 ** 12 // PAGE * PAGE
    t = time.perf_counter()
    assert p.grow(a, far + 5, far + 300) == [] and p.row(a, far // PAGE) == [0, 1, 2]
    p.release_before(a, far + 2 * PAGE)
    assert p.row(a, far // PAGE) == [-1, -1, 2] and p.free_pages == 7
    b = p.fork(a)
    assert p.grow(b, far + 290, far + 400) == [(2, 0)] and p.row(b, far // PAGE + 2) == [0, 1]
    p.release_before(a, far + 4 * PAGE)
    assert p.row(a, far // PAGE) == [-1] * 3 and p.grow(a, far + 6 * PAGE, far + 6 * PAGE + 1) == []
    assert p.row(a, far // PAGE) == [-1] * 6 + [2]
    p.close(a)
    p.close(b)
    assert p.free_pages == 8 and time.perf_counter() - t < 1


def test_a_window_far_on_steps_like_a_young_one():
    """Chunk 10^8 + 2 of a 720p video (pages by the 10^10 before it): as many pages and columns as chunk
    10, which begins at the same token of a page (a chunk is 168.75 pages, and 10 = 10^8 + 2 modulo 4)."""
    got = []
    for first in (10, 10 ** 8 + 2):
        w = PagedWindow(16, 1, 48, 6, 45, 80, window=4, cache_chunks=8, kv_range=8, videos=2, host_only=True)
        t = time.perf_counter()
        a = w.open(first)
        for _ in range(12):
            table, starts, seen = w.layout([a])
            w.slide(a)
        b = w.fork(a)
        w.layout([a, b])
        w.close_video(a)
        got.append((table.shape, len(w.pool.row(b, (w.first_chunk(b) - 8) * w.chunk_tokens // PAGE)), w.pool.free_pages))
        assert time.perf_counter() - t < 5
    assert got[0] == got[1]
