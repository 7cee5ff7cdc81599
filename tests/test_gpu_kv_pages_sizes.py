"""GPU checks of forks and compactions on either side of the sizes from which eight CTAs keep the books instead of one, and of tables in
which a row is several of a warp's pieces, against the rules carried out one page at a time (tests/test_gpu_kv_pages.py)."""
import pytest
import torch

from tests import test_gpu_kv_pages as pages_tests
from tests.test_gpu_kv_pages import tg  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pages,width,room", [
    (6384, 1000, 300),    # pages and entries of both tables together: 16384, and one more
    (6385, 1000, 300),
    (9000, 1111, 900),    # rows of five pieces
    (9000, 256, 7),       # whole pieces
    (20000, 2500, 40),
])
@pytest.mark.parametrize("parents", [[3, 3, 1, -1, 0, 0], [2, 2, 2, 2, 2, 2], [0, 1, 2, 3, -1, 3]])
def test_fork_of_long_rows(tg, pages, width, room, parents):  # noqa: F811
    g = torch.Generator().manual_seed(pages + width)
    page = 16
    cache = pages_tests._cache(tg, pages, 1, page, seed=2)
    refs, table, lens = pages_tests._batch(g, page, pages, 2, 2, min(width - 2, 1000) * page, width)
    pages_tests._check_fork(tg, cache, refs, table, lens, parents, room)
    far = width * page  # as much room as a row can name, for one; what is out of range in a row's last piece
    pages_tests._check_fork(tg, cache, refs, table, lens, [parents[0]], far - lens[parents[0]])
    table[1][width - 1] = pages
    pages_tests._check_fork(tg, cache, refs, table, lens, parents, room, status=tg.ERR_BOUNDS)


def test_fork_of_a_row_that_is_full(tg):  # noqa: F811
    """Every entry is a page, in the last piece too; one that is none there ends the row and is reported."""
    page, width, pages = 16, 1030, 18000
    cache = pages_tests._cache(tg, pages, 1, page, seed=4)
    table = [list(range(i * width, (i + 1) * width)) for i in range(3)]
    refs = [1] * (3 * width) + [0] * (pages - 3 * width)
    lens = [width * page, 1000 * page + 3, 700 * page]
    pages_tests._check_fork(tg, cache, refs, table, lens, [0, 1, 1, 2, 2], 9 * page - 3, status=tg.ERR_BOUNDS)  # (the first has no room)
    table[2][1029], refs[3 * width - 1] = pages, 0
    pages_tests._check_fork(tg, cache, refs, table, lens, [1, 2, 2], 5, status=tg.ERR_BOUNDS)


@pytest.mark.parametrize("pages,batch,count,width", [
    (100, 7000, 7000, 1),     # little, but more sequences than one CTA's shared memory has room for
    (100, 5000, 3000, 0),
    (300, 2000, 2500, 3),
])
def test_fork_of_many_short_rows(tg, pages, batch, count, width):  # noqa: F811
    g = torch.Generator().manual_seed(batch)
    page = 16
    cache = pages_tests._cache(tg, pages, 1, page, seed=3)
    order, refs, table, lens = torch.randperm(pages, generator=g).tolist()[:60], [0] * pages, [], []
    for i in range(batch):
        row = order[i % 20 * width:(i % 20 + 1) * width] if i % 50 == 0 else []
        for p in row:
            refs[p] += 1
        table.append(row + [-1] * (width - len(row)))
        lens.append(len(row) * page - (3 if row else 0))
    parents = torch.randint(-1, batch, (count,), generator=g).tolist()
    parents[:3] = [0, 50, 0]
    if width == 0:
        r, t, n = pages_tests._ints(refs), pages_tests._ints([]).view(batch, 0), pages_tests._ints(lens)
        got = tg.kv_fork(cache, r, t, n, pages_tests._ints(parents))
        assert got[1].shape == (count, 0) and not got[2].any() and got[3].tolist() == [pages] and not got[0].any()
    else:
        pages_tests._check_fork(tg, cache, refs, table, lens, parents, 0)
    pages_tests._status(tg)


@pytest.mark.parametrize("pages,used", [(5192, 3000), (5193, 3000), (4096, 4096), (8192, 8000)])
def test_compact_on_either_side(tg, pages, used):  # noqa: F811
    """Table entries are as many as pages in use, to the next multiple of 300: 8192 pages and entries together, one more, and others."""
    pages_tests.test_compact(tg, pages, used, 16, 64, 1)
