"""What the page oracle refuses: forks of rows that the source does not hold,
and reservations in a row of the table with a gap (CPU)."""
from oracle import pages as op


def copies(refs, table):
    return list(refs), [list(r) for r in table]


def test_fork_of_rows_that_the_source_does_not_hold():
    refs, table = [1, 1, 0, 0, 1], [[0, 1, -1], [4, -1, -1], [-1, -1, -1]]
    before = copies(refs, table)
    for rows in (33, 48):  # a page that is filled in part, and a whole one
        assert op.fork(refs, table, 16, [0], [1], [rows]) == ([[-1, -1]], [0])
        assert (refs, table) == before  # what slot 1 held stays
    pairs, ok = op.fork(refs, table, 16, [0, 0], [1, 2], [40, 17])  # the other entry is served
    assert (pairs, ok) == ([[-1, -1], [1, 2]], [0, 1])
    assert table == [[0, 1, -1], [4, -1, -1], [0, 2, -1]] and refs == [2, 1, 1, 0, 1]
    assert op.fork(refs, table, 16, [0], [1], [0]) == ([[-1, -1]], [1]) and table[1] == [-1, -1, -1]  # no rows: nothing to hold


def test_reserve_in_a_row_with_a_gap():
    refs, table = [1, 0, 1, 1, 0], [[0, -1, 2, -1], [-1, 3, -1, -1]]
    before = copies(refs, table)
    assert op.reserve(refs, table, 16, [0, 1], [48, 17]) == [0, 0]  # pages 2 and 3 would be lost
    assert (refs, table) == before
    assert op.reserve(refs, table, 16, [0, 1], [32, 16]) == [1, 1]  # the pages behind are not reached
    assert table == [[0, 1, 2, -1], [4, 3, -1, -1]] and refs == [1, 1, 1, 1, 1]
