"""The page oracle: worked examples, and what every operation keeps."""
import random

import numpy as np
import pytest

from oracle import pages, rope


def holders(table, lens, pool):
    n = [0] * pool
    for row, m in zip(table, lens):
        for p in row[:pages.held(m)]:
            n[p] += 1
    return n


def test_fork_worked_example():
    # rows: 0 holds pages 3, 1 (70 positions), 1 holds 5 (64), 2 is empty
    table, refs, lens = [[3, 1], [5, -1], [-1, -1]], [0, 1, 0, 1, 0, 1], [70, 64, 0]
    rows, r, n, pairs, short = pages.fork([0, 0, 1], table, refs, lens)
    # page 1 is shared by rows 0 and 1: row 1 gets a copy in page 0; page 5 (full) passes to row 2
    assert rows == [[3, 1], [3, 0], [5, -1]] and n == [70, 70, 64] and pairs == [(1, 0)] and not short
    assert r == [1, 1, 0, 2, 0, 1]
    # somebody else holds page 1 too: both rows get copies
    rows, r, n, pairs, short = pages.fork([0, 0, -1], table, [0, 2, 0, 1, 0, 1], lens)
    assert rows == [[3, 0], [3, 2], [-1, -1]] and n == [70, 70, 0] and pairs == [(1, 0), (1, 2)]
    assert r == [1, 1, 1, 2, 0, 0]
    # no page left: the row keeps its whole pages
    rows, r, n, pairs, short = pages.fork([0, 0], [[0, 1], [2, -1]], [1, 1, 2], [70, 64])
    assert rows == [[0, 1], [0, -1]] and n == [70, 64] and short == [1] and r == [2, 1, 1]


def test_resize_worked_example():
    table, refs, lens = [[3, 1, -1], [3, 1, -1], [5, 0, 2]], [1, 2, 1, 2, 0, 1], [100, 100, 130]
    rows, r, n, pairs, short = pages.resize(table, refs, lens, [101, 129, 60])
    # row 2 gives back pages 0 and 2; row 0 keeps page 1, row 1 gets a copy in 0 and a new page 2
    assert rows == [[3, 1, -1], [3, 0, 2], [5, -1, -1]] and n == [101, 129, 60] and pairs == [(1, 0)] and not short
    assert r == [1, 1, 1, 2, 0, 1]
    rows, r, n, pairs, short = pages.resize([[0, -1], [1, -1]], [1, 1, 0], [64, 64], [128, 128])
    assert rows == [[0, 2], [1, -1]] and n == [128, 64] and short == [1] and r == [1, 1, 1]


def test_compact_worked_example():
    rows, r, to, n, pairs = pages.compact([[4, 6], [2, 9]], [0, 0, 1, 0, 1, 0, 3], [128, 10])
    assert n == 3 and pairs == [(4, 0), (6, 1)] and rows == [[0, 1], [2, 9]]
    assert to == [-1, -1, 2, -1, 0, -1, 1] and r == [1, 3, 1, 0, 0, 0, 0]


@pytest.mark.parametrize("seed", range(20))
def test_what_every_operation_keeps(seed):
    """Counts stay the holders plus the other owners; partly filled pages that may be written have one holder; what a
    page holds is moved, never lost."""
    rng = random.Random(seed)
    batch, width, pool = rng.randint(1, 6), 4, 40
    other = [0] * pool
    for p in rng.sample(range(pool), 3):
        other[p] = 1
    table, lens = [[-1] * width for _ in range(batch)], [0] * batch
    refs = list(other)
    content = [None] * pool          # what a page holds: (row's tokens)
    logical = [[] for _ in range(batch)]
    stamp = 0

    def check():
        n = holders(table, lens, pool)
        assert refs == [a + b for a, b in zip(n, other)]
        for row, m, want in zip(table, lens, logical):
            got = [x for t in range(pages.held(m)) for x in content[row[t]]][:m]
            assert got == want

    for _ in range(12):
        op = rng.choice(["fork", "resize", "resize", "compact"])
        if op == "fork":
            parent = [rng.randint(-1, batch - 1) for _ in range(batch)]
            table, refs, lens, pairs, short = pages.fork(parent, table, refs, lens)
            logical = [list(logical[p]) if p >= 0 else [] for p in parent]
        elif op == "resize":
            new = [rng.choice([0, n, max(0, n - 1), min(256, n + 1), rng.randint(0, 200)]) for n in lens]
            old = lens
            table, refs, lens, pairs, short = pages.resize(table, refs, lens, new)
        else:
            table, refs, to, _, pairs = pages.compact(table, refs, lens)
            moved = [0] * pool
            for p in range(pool):
                if to[p] >= 0:
                    moved[to[p]] = other[p]
            other = moved
        before = list(content)
        for src, dst in pairs:
            content[dst] = list(before[src]) if before[src] else None
        if op == "resize":
            assert not short
            for b in range(batch):
                logical[b] = logical[b][:lens[b]]
                for p in range(old[b], lens[b]):
                    page = table[b][p // 64]
                    assert refs[page] == 1
                    if p % 64 == 0 or content[page] is None:
                        content[page] = [None] * 64
                    content[page][p % 64] = stamp
                    logical[b].append(stamp)
                    stamp += 1
        check()


def test_rope_axes_reduces_to_one_axis():
    rng = np.random.default_rng(0)
    x, pos = rng.normal(size=(5, 128)), np.arange(5) * 1000
    for pairing in (0, 1):
        one = rope.apply_rope(x, pos, 1e4, pairing)
        assert np.array_equal(rope.apply_rope_axes(x, pos[None], [0] * 64, 1e4, pairing), one)
        axis = [j % 3 for j in range(64)]
        assert np.array_equal(rope.apply_rope_axes(x, np.stack([pos] * 3), axis, 1e4, pairing), one)
        # a pair keeps its length; an axis at position 0 leaves its blocks alone
        got = rope.apply_rope_axes(x, np.stack([pos, 0 * pos, pos]), axis, 1e4, pairing)
        for j, (a, b) in enumerate(rope.block_dims(128, pairing)):
            assert np.allclose(np.hypot(got[:, a], got[:, b]), np.hypot(x[:, a], x[:, b]), rtol=1e-12)
            if axis[j] == 1:
                assert np.array_equal(got[:, [a, b]], x[:, [a, b]])
