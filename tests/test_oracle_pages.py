"""The page oracle's own pins: hand cases, and counts that stay the tables' (CPU)."""
import random

from oracle import pages as op


def counts(table, n):
    c = [0] * n
    for row in table:
        for p in row:
            if 0 <= p < n:
                c[p] += 1
    return c


def test_hand_cases():
    refs, table = [0] * 6, [[-1] * 4 for _ in range(3)]
    assert op.reserve(refs, table, 16, [1, 0], [33, 16]) == [1, 1]
    assert table == [[3, -1, -1, -1], [0, 1, 2, -1], [-1] * 4] and refs == [1, 1, 1, 1, 0, 0]
    assert op.reserve(refs, table, 16, [0, 2], [64, 20]) == [0, 1]  # three more do not fit, two do
    assert table[2] == [4, 5, -1, -1]
    op.release(refs, table, 16, [2], [0])
    pairs, ok = op.fork(refs, table, 16, [1], [2], [40])
    assert (pairs, ok) == ([[2, 4]], [1]) and table[2] == [0, 1, 4, -1] and refs == [2, 2, 1, 1, 1, 0]
    op.release(refs, table, 16, [0, 1], [0, 0])
    assert refs == [1, 1, 0, 0, 1, 0]
    assert op.compact(refs, table, 3) == [(4, 2), (-1, -1), (-1, -1)] and table[2] == [0, 1, 2, -1] and refs == [1, 1, 1, 0, 0, 0]


def test_fork_without_pages_leaves_the_slot_empty():
    refs, table = [1, 1, 1], [[0, 1], [2, -1], [-1, -1]]
    pairs, ok = op.fork(refs, table, 16, [0, 0], [2, 1], [20, 20])
    assert ok == [1, 0] and pairs == [[1, 2], [-1, -1]]  # the page that slot 1 let go serves slot 2
    assert table == [[0, 1], [-1, -1], [0, 2]] and refs == [2, 1, 1]


def test_counts_stay_the_tables():
    rnd = random.Random(7)
    for _ in range(60):
        n, S, W, page = rnd.randint(1, 40), rnd.randint(1, 8), rnd.randint(1, 9), 16
        refs, table = [0] * n, [[-1] * W for _ in range(S)]
        for _ in range(12):
            k = rnd.randint(0, 5)
            seq = [rnd.randint(-1, S) for _ in range(k)]
            rows = [rnd.randint(-3, W * page + 5) for _ in range(k)]
            what = rnd.randint(0, 3)
            if what == 0:
                op.reserve(refs, table, page, seq, rows)
            elif what == 1:
                op.fork(refs, table, page, seq, [rnd.randint(-1, S) for _ in range(k)], rows)
            elif what == 2:
                op.release(refs, table, page, seq, rows)
            else:
                before = [[p for p in row if p >= 0] for row in table]
                m = rnd.randint(1, 20)
                pairs = op.compact(refs, table, m)
                to = {a: b for a, b in pairs if a >= 0}
                assert len(to) == len([a for a, _ in pairs if a >= 0]) and not set(to) & set(to.values())
                assert [[to.get(p, p) for p in row] for row in before] == [[p for p in row if p >= 0] for row in table]
                if m >= n // 2:
                    used = sum(c > 0 for c in refs)
                    assert all(c > 0 for c in refs[:used])
            assert refs == counts(table, n)
