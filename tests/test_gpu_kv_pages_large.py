"""GPU checks of forks whose tables are so large that the pages they ask for, added up, pass 32 bits. Tables of some ten
gigabytes of entries, nearly all of which say that there is no page."""
import pytest
import torch

from tests.test_gpu_kv_pages import _bytes, _cache, _ints, _status, tg  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pages,count,width", [
    (40, 18, 2 ** 27 - 1),      # more than 2^31 within a warp
    (40, 1100, 2 ** 21),        # within the first 1024 sequences
    (20000, 1100, 2 ** 21),
])
def test_needs_that_add_up_to_more_than_32_bits(tg, pages, count, width):  # noqa: F811
    """Every sequence asks for all the pages that its row of the table can name. The first gets what there is; entries
    of later ones come after 2^31 others, and are none. The last but one continues a sequence whose open page another
    holds: its tokens have no page to go to."""
    page = 16
    cache = _cache(tg, pages, 1)
    before = _bytes(cache)
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[3] = 2
    table = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
    table[0, 0] = 3
    parents = [-1] * count
    parents[count - 2] = 0
    out = (torch.empty_like(refs), torch.full((count, width), 7, dtype=torch.int32, device="cuda"), torch.empty(count, dtype=torch.int32, device="cuda"), _ints([9]))
    got = tg.kv_fork(cache, refs, table, _ints([5]), _ints(parents), room=(width - 1) * page + 1, out=out)
    _status(tg)
    free = [p for p in range(pages) if p != 3]
    want = count * width - (pages - 1)                     # that are lacking
    assert got[3].tolist() == [max(-want, -2 ** 31)]
    assert got[0].tolist() == [1] * pages                  # page 3: its other holder's
    assert got[2].tolist() == [5 if i == count - 2 else 0 for i in range(count)]
    assert got[1][0, :pages - 1].tolist() == free
    got[1][0, :pages - 1] = -1
    for rows in got[1].split(max(1, 2 ** 28 // width)):
        assert int(rows.max()) == int(rows.min()) == -1
    for a, b in zip(_bytes(cache), before):
        assert torch.equal(a, b)
