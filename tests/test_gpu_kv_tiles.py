"""GPU checks of the cache attention's kernel for many rows where its look-ahead (pages of four tiles of 128 keys at a time,
codes in pieces of 8 KB, copies as large as a page allows) can go wrong: every page size, segments of few and of many tiles,
ends inside a piece, pages that are missing. Against the definition in float64, with tests/kv_reference.py's tolerances."""
import pytest
import torch

from tests import kv_reference as ref
from tests.test_gpu_attention_kv import _case, _check, _ints, _status_ok, tg  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ct,dt", [(0, 1), (1, 0)])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_every_page_size(tg, page, dim, ct, dt):  # noqa: F811
    counts, lens = [70, 129, 1, 0, 65, 300], [3001, 129, 1, 77, 640, 1555]
    cache, host, table, q = _case(tg, counts, lens, page, 2, 4, dim, ct, dt, seed=page + dim)
    cu = [0] + torch.tensor(counts).cumsum(0).tolist()
    for causal, window in ((True, 0), (True, 1000), (False, 0)):
        args = (q.cuda(), cache, table.cuda(), _ints(lens), _ints(cu))
        out, lse = tg.attention_kv(*args, max_new=300, max_len=3001, causal=causal, window=window, return_lse=True)
        _check(out, lse, host, table, q, counts, lens, page, causal, window, dim ** -0.5)
        assert torch.equal(out, tg.attention_kv(*args, max_new=300, max_len=3001, causal=causal, window=window))
    _status_ok(tg)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_pages_that_are_missing(tg, page, dim):  # noqa: F811
    """At the beginning, in the middle of a tile and of the four, at the end: reported, their keys left out, the others seen."""
    n, length = 80, 2 * 1024 + 3 * 16 + 5
    cache, host, table, q = _case(tg, [n], [length], page, 1, 2, dim, 0, 0, seed=7)
    slots = -(-length // page)
    hidden = sorted({0, slots // 3, slots // 2, slots // 2 + 1, slots - 1})
    bad = table.clone()
    bad[0, hidden] = torch.tensor([-1, 2 ** 31 - 1, host[0].shape[0], -2 ** 31, -1], dtype=torch.int32)[:len(hidden)]
    out, lse = tg.attention_kv(q.cuda(), cache, bad.cuda(), _ints([length]), _ints([0, n]), max_new=n, max_len=length, causal=False, return_lse=True)
    assert tg.tg_device_status(None)[0] == tg.ERR_BOUNDS
    seen = [i for i in range(slots) if i not in hidden]
    k, v = (torch.cat([ref.gather(c, s, table[0, [i]].long(), min(page, length - i * page)) for i in seen]) for c, s in ((host[0], host[2]), (host[1], host[3])))
    o, want, tol, ltol = ref.attention(q.double(), k, v, len(k), False, 0, dim ** -0.5)
    ref.near(out, o, tol + o.abs() * ref.half_step(out.dtype) + 2.0 ** -25)
    ref.near(lse, want, ltol)
    _status_ok(tg)


def test_more_sequences_than_a_share_has_tiles(tg):  # noqa: F811
    """Segments of one tile: the look-ahead passes over sequences, and over ones without rows."""
    g = torch.Generator().manual_seed(3)
    lens = [int(x) for x in torch.randint(1, 260, (500,), generator=g)]
    counts = [0 if i % 7 == 3 else min(x, 33 + i % 40) for i, x in enumerate(lens)]
    for dim in (64, 128):
        cache, host, table, q = _case(tg, counts, lens, 32, 1, 2, dim, 1, 0, seed=dim)
        cu = [0] + torch.tensor(counts).cumsum(0).tolist()
        out, lse = tg.attention_kv(q.cuda(), cache, table.cuda(), _ints(lens), _ints(cu), max_new=72, max_len=260, return_lse=True)
        _check(out, lse, host, table, q, counts, lens, 32, True, 0, dim ** -0.5)
    _status_ok(tg)
