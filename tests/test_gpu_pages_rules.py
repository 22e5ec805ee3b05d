"""Page calls that would lose rows or pages: forks of rows that the source does
not hold, reservations in a row of the table with a gap, and sequences that are
cut back into a page which others hold too."""
import random

import pytest

from oracle import pages as op

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import moe_speculative_decoding_router_amd as m  # noqa: E402
from test_gpu_pages import DEV, Pool, dev  # noqa: E402


def pool_of(refs, table, page=16):
    p = Pool(len(refs), len(table), len(table[0]), page)
    p.refs, p.table = list(refs), [list(r) for r in table]
    p.drefs, p.dtable = dev(p.refs), dev(p.table)
    return p


def test_fork_of_rows_that_the_source_does_not_hold():
    p = pool_of([1, 1, 0, 0, 1], [[0, 1, -1], [4, -1, -1], [-1, -1, -1]])
    assert p.fork([0], [1], [33]) == [0] and p.table[1] == [4, -1, -1]
    assert p.fork([0], [1], [48]) == [0]
    assert p.fork([0, 0], [1, 2], [40, 17]) == [0, 1]
    assert p.fork([0], [1], [0]) == [1]
    p = pool_of([1, 1], [[0, 2, 1], [-1, -1, -1], [-1, -1, -1]])  # an entry outside the pool holds no page
    assert p.fork([0, 0], [1, 2], [48, 16]) == [0, 1]


@pytest.mark.parametrize("at", [0, 63, 64, 255, 256, 700, 799, None])
@pytest.mark.parametrize("part", [False, True])
def test_one_missing_page_of_a_long_source(at, part):
    """The missing entry lies in any pass of the search, or is the one filled in part."""
    W, page = 801, 16
    row = list(range(W))
    if at is not None:
        row[at] = -1
    refs = [int(p in row) for p in range(W)] + [0] * 900
    p = pool_of(refs, [row, [-1] * W, [-1] * W], page)
    rows = 800 * page + (7 if part else 0)
    assert p.fork([0, 0], [2, 1], [rows, 16 * (at or 0)]) == [int(at is None), 1]
    if part:
        p = pool_of(refs, [row[:800] + [-1], [-1] * W, [-1] * W], page)
        assert p.fork([0], [1], [rows]) == [0]


@pytest.mark.parametrize("gap,behind", [(0, 1), (1, 799), (62, 64), (63, 65), (300, 301), (700, 799)])
def test_reserve_in_a_row_with_a_gap(gap, behind):
    """Nothing is taken where a page behind the gap would be overwritten; entries of the list around it are served."""
    W, page = 801, 16
    row = list(range(gap)) + [-1] * (W - gap)
    row[behind] = behind
    refs = [int(p in row) for p in range(W)] + [0] * 900
    p = pool_of(refs, [[-1] * W, row, [-1] * W], page)
    assert p.reserve([0, 1, 2], [40, page * 800, 33]) == [1, 0, 1]
    assert p.reserve([1], [page * behind]) == [1]  # the gap filled up to the page behind it
    assert p.reserve([1], [page * 801]) == [1]
    counts = [0] * len(p.refs)
    for r in p.table:
        for x in r:
            if x >= 0:
                counts[x] += 1
    assert counts == p.refs


@pytest.mark.parametrize("seed", range(6))
def test_random_tables_with_gaps(seed):
    """Tables of any entries, counts that are theirs: after every call they still are, and equal to the oracle's."""
    rnd = random.Random(seed)
    P, S, W, page = rnd.choice([30, 400]), rnd.randint(2, 20), rnd.choice([3, 70, 130]), 16
    table = [[rnd.choice([-1, rnd.randint(-2, P + 2)]) for _ in range(W)] for _ in range(S)]
    refs = [0] * P
    for r in table:
        for x in r:
            if 0 <= x < P:
                refs[x] += 1
    p = pool_of(refs, table, page)
    for _ in range(20):
        k = rnd.randint(1, 20)
        names, rows = [rnd.randint(-1, S) for _ in range(k)], [rnd.randint(0, W * page) // rnd.choice([1, 9, 60]) for _ in range(k)]
        what = rnd.randint(0, 3)
        if what == 0:
            p.reserve(names, rows)
        elif what == 1:
            p.fork([rnd.randint(0, S // 2) for _ in range(k)], [rnd.randint(S // 4, S) for _ in range(k)], rows)
        elif what == 2:
            p.release(names[:3], rows[:3])
        else:
            p.compact(rnd.choice([None, 2]))
        counts = [0] * P
        for r in p.table:
            for x in r:
                if 0 <= x < P:
                    counts[x] += 1
        assert counts == p.refs


@pytest.mark.parametrize("who", [0, 1])
@pytest.mark.parametrize("keep", [0, 5, 16, 20, 32, 40])
def test_cut_back_into_a_shared_page(keep, who):
    """A prompt of 40 rows and its fork: one of the two is cut back below the fork's rows and continued, as the
    header describes, in a slot of its own.  The other's rows stay what they were."""
    page, n, more = 16, 40, 9
    g = torch.Generator(device=DEV).manual_seed(keep + who)
    p = Pool(30, 4, 6, page)
    cache = m.kv4_cache(30, page, 2, 64, device=DEV)
    rows = torch.randn((2, n + more, 2, 64), generator=g, device=DEV)
    append = lambda slot, a, b, at: m.kv4_append(cache, rows[0, a:b], rows[1, a:b], p.dtable[slot:slot + 1].contiguous(),  # noqa: E731
                                                 dev([at]), [0, b - a], return_stored=True)[0]
    read = lambda slot, r: m.kv4_read(cache, p.dtable[slot:slot + 1].contiguous(), dev([0]), [0, r], dtype=torch.float32)[0]  # noqa: E731
    p.reserve([0], [n])
    stored = append(0, 0, n, 0)
    pairs, ok = m.kv4_fork(p.drefs, p.dtable, page, dev([0]), dev([1]), dev([n]))
    assert op.fork(p.refs, p.table, page, [0], [1], [n]) == (pairs.tolist(), ok.tolist())
    m.kv4_copy_pages(cache, pairs)
    p.release([who], [keep])
    # continued in slot 2
    pairs, ok = m.kv4_fork(p.drefs, p.dtable, page, dev([who]), dev([2]), dev([keep]))
    assert op.fork(p.refs, p.table, page, [who], [2], [keep]) == (pairs.tolist(), ok.tolist()) and ok.tolist() == [1]
    m.kv4_copy_pages(cache, pairs)
    p.release([who], [0])
    p.reserve([2], [keep + more])
    written = {p.table[2][j] for j in range(keep // page, -(-(keep + more) // page))}
    assert all(p.refs[x] == 1 for x in written)
    own = append(2, n, n + more, keep)
    assert torch.equal(read(2, keep + more), torch.cat([stored[:keep], own]))
    assert torch.equal(read(1 - who, n), stored)
