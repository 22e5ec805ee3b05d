"""Page calls that would lose rows or pages: forks of rows that the source does
not hold."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

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
