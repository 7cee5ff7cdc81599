"""GPU checks of pages copied, forked, given, let go of and compacted, against the rules carried out one page at a
time on the CPU. Everything here is whole numbers and codes that are moved: equal, or wrong."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import tiled_tensor_core_tcgen05_gb300 as m
    torch.cuda.set_device(0)
    return m


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _status(tg, want=None):
    st, where = tg.tg_device_status(None)
    assert st == (tg.OK if want is None else want), f"device status {st} at {where}"


def _cache(tg, pages, kv=2, page=16, dim=64, dtype=torch.int8, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    k, v = (torch.randint(-100, 101, (pages, kv, page, dim), generator=g, device="cuda").float().to(dtype) for _ in range(2))
    return tg.KvCache(k, v, *(torch.rand(pages, kv, generator=g, device="cuda") for _ in range(2)))


def _bytes(cache):
    return [t.clone().view(torch.uint8).cpu() if t.dtype is not torch.float32 else t.clone().cpu() for t in cache.args]


def fork(refs, table, lens, parents, page, room):
    """(refs, table, lens, spare, copies): copies are (from, to, tokens)."""
    refs, width, count = list(refs), len(table[0]) if table else 0, {}
    pages = len(refs)
    held = []
    for row in table:
        h = []
        for p in row:
            if not 0 <= p < pages:
                break
            h.append(p)
        held.append(h)
    lens = [n if 0 <= n <= len(h) * page else 0 for n, h in zip(lens, held)]
    before = list(refs)
    for h in held:
        for p in h:
            refs[p] -= 1
    rows, sources, out_lens, done = [], [], [], set()
    for p in parents:
        if not 0 <= p < len(held):
            rows.append([])
            sources.append(None)
            out_lens.append(0)
            continue
        n, h = lens[p], held[p]
        row = h[:n // page]
        if p not in done:
            for q in h[n // page:]:
                if before[q] != 1:
                    break
                row.append(q)
        done.add(p)
        sources.append(h[n // page] if n % page and len(row) == n // page else None)
        rows.append(row)
        out_lens.append(n)
        for q in row:
            refs[q] += 1
    free = [p for p in range(pages) if refs[p] == 0 and p not in sources]
    copies, lacking = [], 0
    for i, (row, n) in enumerate(zip(rows, out_lens)):
        for at in range(len(row), min(width, -(-(n + room) // page))):
            if not free:
                lacking += 1
                continue
            q = free.pop(0)
            refs[q] += 1
            if sources[i] is not None and at == n // page:
                copies.append((sources[i], q, n % page))
            row.append(q)
    return refs, [row + [-1] * (width - len(row)) for row in rows], out_lens, len(free) - lacking, copies


def after(state, copies):
    k, v, ks, vs = (t.clone() for t in state)
    for a, b, n in copies:
        for to, of in ((k, state[0]), (v, state[1])):
            to[b, :, :n] = of[a, :, :n]
        ks[b], vs[b] = state[2][a], state[3][a]
    return [k, v, ks, vs]


def _check_fork(tg, cache, refs, table, lens, parents, room, out=None, status=None):
    page, before = cache.page, _bytes(cache)
    want = fork(refs, table, lens, range(len(lens)) if parents is None else parents, page, room)
    width = len(table[0]) if table else 0
    args = [_ints(refs), _ints(table).view(len(table), width), _ints(lens)]
    got = tg.kv_fork(cache, *args, None if parents is None else _ints(parents), room=room, out=out)
    _status(tg, status)
    assert got[0].tolist() == want[0], "refs"
    assert got[1].tolist() == want[1], "table"
    assert got[2].tolist() == want[2], "lens"
    assert got[3].tolist() == [want[3]], "spare"
    for a, b in zip(_bytes(cache), after(before, want[4])):
        assert torch.equal(a, b)
    assert args[0].tolist() == list(refs) and args[1].tolist() == [list(r) for r in table] and args[2].tolist() == list(lens)
    return got, want


def _batch(g, page, pages, prompts, beams, longest, width):
    """Sequences that share their prompt's full pages, a consistent refs, in pages in no order."""
    order = torch.randperm(pages, generator=g).tolist()
    refs, table, lens = [0] * pages, [], []
    for _ in range(prompts):
        prompt, whole = sorted(torch.randint(0, longest + 1, (2,), generator=g).tolist())
        shared = [order.pop() for _ in range(prompt // page)]
        for _ in range(beams):
            row = shared + [order.pop() for _ in range(-(-whole // page) - len(shared))]
            for p in row:
                refs[p] += 1
            table.append(row + [-1] * (width - len(row)))
            lens.append(whole)
    return refs, table, lens


@pytest.mark.parametrize("page,dim,kv,dtype", [(16, 64, 1, torch.int8), (32, 128, 3, torch.float8_e4m3fn), (64, 64, 2, torch.float8_e4m3fn), (128, 128, 2, torch.int8)])
@pytest.mark.parametrize("prompts,beams,room", [(1, 1, 0), (1, 4, 1), (3, 5, 0), (7, 3, 40), (40, 2, 1)])
def test_fork_of_random_parents(tg, page, dim, kv, dtype, prompts, beams, room):
    g = torch.Generator().manual_seed(page + prompts)
    pages = prompts * beams * 12 + 5
    cache = _cache(tg, pages, kv, page, dim, dtype)
    refs, table, lens = _batch(g, page, pages, prompts, beams, 5 * page, 9)
    n = len(lens)
    for parents in (None, torch.randint(-1, n, (n,), generator=g).tolist(), [0] * n, [-1] * n, list(range(n))[::-1], torch.randint(0, n, (2 * n + 1,), generator=g).tolist()):
        _check_fork(tg, cache, refs, table, lens, parents, room)


def test_fork_step_after_step(tg):
    """A search of many steps on its own results: nothing is lost and nothing given twice."""
    g = torch.Generator().manual_seed(3)
    page, pages, n = 16, 60, 6
    cache = _cache(tg, pages)
    refs, table, lens = [0] * pages, [[-1] * 12 for _ in range(n)], [0] * n
    (r, t, ln, _), _ = _check_fork(tg, cache, refs, table, lens, None, 21)
    for step in range(40):
        ln = (ln + torch.randint(1, 6, (1,), generator=g).item()).clamp(max=int((t >= 0).sum(1).min()) * page)
        parents = torch.randint(0, n, (n,), generator=g).tolist() if step % 3 else None
        (r, t, ln, spare), _ = _check_fork(tg, cache, r.tolist(), t.tolist(), ln.tolist(), parents, 5)
        entries = t[t >= 0]
        assert torch.equal(torch.bincount(entries.long(), minlength=pages).int(), r)
        assert int(spare) == int((r == 0).sum())
        if step % 10 == 9:  # let everything go, and begin again
            (r, t, ln, spare), _ = _check_fork(tg, cache, r.tolist(), t.tolist(), ln.tolist(), [-1] * n, 21)


def test_fork_where_pages_are_lacking(tg):
    cache = _cache(tg, 6)
    refs, table, lens = [1, 1, 0, 0, 0, 1], [[0, 1, 5, -1, -1]], [40]
    got, _ = _check_fork(tg, cache, refs, table, lens, [0, 0, 0, 0, 0], 9)
    assert int(got[3]) == 3 - 9  # 49 tokens are 4 pages: one for the first child, two for each of the four others
    _check_fork(tg, cache, refs, table, lens, [0, -1, 0], 1000000, status=tg.ERR_BOUNDS)  # room stops at the table's width


def test_fork_copies_no_page_that_is_given_away(tg):
    """Two sequences hold the same open page: neither keeps it, both get copies, and it is free only afterwards."""
    cache = _cache(tg, 4)
    refs, table, lens = [2, 0, 0, 2], [[3, 0], [3, 0]], [20, 20]
    got, want = _check_fork(tg, cache, refs, table, lens, [0, 1], 0)
    assert want[1] == [[3, 1], [3, 2]] and want[0] == [0, 1, 1, 2]
    # another holder (a cache of prompts) keeps pages: an open one stays as it is
    _check_fork(tg, cache, [2, 0, 0, 2], [[3, 0]], [20], [0], 0)


def test_fork_sizes_at_the_ends(tg):
    cache = _cache(tg, 5)
    _check_fork(tg, cache, [0] * 5, [[-1, -1]], [0], [], 3)                       # no new sequence
    got = tg.kv_fork(cache, _ints([0] * 5), _ints([]).view(0, 3), _ints([]), _ints([-1, -1]), room=17)  # no old one
    assert got[1].tolist() == [[0, 1, -1], [2, 3, -1]] and got[3].tolist() == [1]
    got = tg.kv_fork(cache, _ints([0] * 5), _ints([[], []]).view(2, 0), _ints([0, 0]), _ints([1, 0]))  # no place for a page
    assert got[1].shape == (2, 0) and got[2].tolist() == [0, 0] and got[3].tolist() == [5]
    _status(tg)
    none = _cache(tg, 0)
    got = tg.kv_fork(none, _ints([]), _ints([[-1]]), _ints([0]), _ints([0]), room=1)
    assert got[1].tolist() == [[-1]] and got[3].tolist() == [-1]
    _status(tg)


def test_fork_of_many_sequences_and_long_tables(tg):
    """More sequences than threads of a CTA, rows longer than a warp's piece, pools of many pages."""
    g = torch.Generator().manual_seed(1)
    page, n, width, pages = 16, 1500, 3, 9001
    cache = _cache(tg, pages, 1)
    refs, table, lens = _batch(g, page, pages, n // 3, 3, 2 * page + 5, width)
    _check_fork(tg, cache, refs, table, lens, torch.randint(-1, len(lens), (2100,), generator=g).tolist(), 3)
    cache = _cache(tg, 5000, 1)
    refs, table, lens = _batch(g, page, 5000, 1, 4, 700 * page, 1111)
    _check_fork(tg, cache, refs, table, lens, [3, 3, 1, -1, 0, 0], 900)


def test_fork_out_of_range(tg):
    cache = _cache(tg, 8)
    refs, table, lens = [1, 1, 1, 1, 0, 0, 0, 0], [[0, 1, -1], [2, 3, -1]], [20, 25]
    _check_fork(tg, cache, refs, table, lens, [1, 2, 0], 0, status=tg.ERR_BOUNDS)             # no such parent
    _check_fork(tg, cache, refs, table, [20, 33], [1, 0, 1], 0, status=tg.ERR_BOUNDS)         # longer than its pages
    _check_fork(tg, cache, refs, table, [-1, 20], [1, 0, 0], 0, status=tg.ERR_BOUNDS)
    _check_fork(tg, cache, refs, [[0, 8, 1], [2, 3, -1]], [16, 25], [0, 0, 1], 2, status=tg.ERR_BOUNDS)  # no such page
    _status(tg)


def test_fork_into_given_tensors_on_a_stream_and_in_a_graph(tg):
    page = 16
    cache, other = _cache(tg, 20), _cache(tg, 20)
    refs, table, lens = [2, 1, 1] + [0] * 17, [[0, 1, -1, -1], [0, 2, -1, -1]], [20, 20]
    out = tuple(torch.full(s, 77, dtype=torch.int32, device="cuda") for s in ((20,), (3, 4), (3,), (1,)))
    version = cache.k._version
    got, _ = _check_fork(tg, cache, refs, table, lens, [1, 1, 0], 30, out=out)
    assert all(a is b for a, b in zip(got, out)) and cache.k._version > version
    r, t, n, p = _ints(refs), _ints(table), _ints(lens), _ints([1, 1, 0])
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            made = tg.kv_fork(other, r, t, n, p, room=30)
    for parents in ([1, 1, 0], [0, 0, 0], [-1, 1, 0]):
        p.copy_(_ints(parents))
        before = _bytes(other)
        want = fork(refs, table, lens, parents, page, 30)
        graph.replay()
        torch.cuda.synchronize()
        assert [x.tolist() for x in made] == [want[0], want[1], want[2], [want[3]]]
        for a, b in zip(_bytes(other), after(before, want[4])):
            assert torch.equal(a, b)
    _status(tg)


@pytest.mark.parametrize("pages,used,page,dim,kv", [(1, 0, 16, 64, 1), (1, 1, 16, 64, 1), (2, 1, 128, 128, 1), (33, 20, 16, 64, 3), (300, 7, 32, 64, 2), (9000, 4000, 16, 64, 1),
                                                    (20011, 19000, 16, 64, 1)])
def test_compact(tg, pages, used, page, dim, kv):
    g = torch.Generator().manual_seed(pages)
    cache = _cache(tg, pages, kv, page, dim, torch.float8_e4m3fn if pages % 2 else torch.int8)
    held = sorted(torch.randperm(pages, generator=g)[:used].tolist())
    refs = [0] * pages
    for p in held:
        refs[p] = int(torch.randint(1, 4, (1,), generator=g))
    width = 300 if used > 1000 else 5
    entries = [held[i] if held and i < len(held) * 9 // 10 else -1 for i in torch.randperm(max(used, 1), generator=g).tolist()]
    entries += [-1] * (-len(entries) % width)
    table = [entries[i:i + width] for i in range(0, len(entries), width)]
    before = _bytes(cache)
    got = tg.kv_compact(cache, _ints(refs), _ints(table))
    _status(tg)
    where = list(range(pages))
    for b, a in zip([p for p in range(used) if not refs[p]], [p for p in held if p >= used]):
        where[a] = b
    where = [w if refs[p] else -1 for p, w in enumerate(where)]
    new = [0] * pages
    for p in held:
        new[where[p]] = refs[p]
    assert got[0].tolist() == new and got[2].tolist() == where and got[3].tolist() == [used]
    assert got[1].tolist() == [[where[p] if p >= 0 else -1 for p in row] for row in table]
    state = _bytes(cache)
    want = after(before, [(p, where[p], page) for p in held if where[p] != p])
    assert all(torch.equal(a, b) for a, b in zip(state, want))


def test_compact_of_a_page_nobody_holds_and_of_none_there_is(tg):
    cache = _cache(tg, 4)
    got = tg.kv_compact(cache, _ints([0, 1, -3, 1]), _ints([[1, 2, 3, 4]]))
    assert got[1].tolist() == [[1, -1, 0, -1]] and got[0].tolist() == [1, 1, 0, 0]
    _status(tg, tg.ERR_BOUNDS)


@pytest.mark.parametrize("page,dim,kv,dtype", [(16, 64, 1, torch.int8), (32, 128, 3, torch.float8_e4m3fn), (128, 128, 8, torch.int8)])
def test_copy(tg, page, dim, kv, dtype):
    g = torch.Generator().manual_seed(page)
    a, b = _cache(tg, 40, kv, page, dim, dtype), _cache(tg, 55, kv, page, dim, dtype, seed=1)
    src, dst = torch.randint(0, 40, (30,), generator=g), torch.randperm(55, generator=g)[:30]
    before, of = _bytes(b), _bytes(a)
    assert tg.kv_copy(a, src.int().cuda(), dst.int().cuda(), to=b) is None
    want = before
    for x, y in zip(want, of):
        x[dst] = y[src]
    assert all(torch.equal(x, y) for x, y in zip(_bytes(b), want)) and all(torch.equal(x, y) for x, y in zip(_bytes(a), of))
    tg.kv_copy(a, _ints([3, 7, 9]), _ints([4, 7, 0]))  # within a cache; a page to itself
    for x in of:
        x[[4, 7, 0]] = x[[3, 7, 9]].clone()
    assert all(torch.equal(x, y) for x, y in zip(_bytes(a), of))
    tg.kv_copy(a, _ints([]), _ints([]))
    _status(tg)
    tg.kv_copy(a, _ints([40, 2, -1, 5]), _ints([1, 55, 3, 6]), to=b)  # left out: no such page
    for x, y in zip(want, of):
        x[6] = y[5]
    assert all(torch.equal(x, y) for x, y in zip(_bytes(b), want))
    _status(tg, tg.ERR_BOUNDS)


def test_refusals(tg):
    cache = _cache(tg, 4)
    r, t, n = _ints([0] * 4), _ints([[-1, -1]]), _ints([0])
    with pytest.raises(ValueError, match="refs must have shape"):
        tg.kv_fork(cache, r[:3], t, n)
    with pytest.raises(ValueError, match="lens must have shape"):
        tg.kv_fork(cache, r, t, _ints([0, 0]))
    with pytest.raises(TypeError, match="int32"):
        tg.kv_fork(cache, r.long(), t, n)
    with pytest.raises(ValueError, match="parents"):
        tg.kv_fork(cache, r, t, n, _ints([[0]]))
    with pytest.raises(TypeError, match="CUDA"):
        tg.kv_fork(cache, r, t, n, torch.zeros(1, dtype=torch.int32))
    with pytest.raises(tg.TgError, match="room"):
        tg.kv_fork(cache, r, t, n, room=-1)
    with pytest.raises(tg.TgError, match="overlaps"):
        tg.kv_fork(cache, r, t, n, out=(r, t.clone(), n.clone(), _ints([0])))
    with pytest.raises(tg.TgError, match="overlaps"):
        tg.kv_fork(cache, r, t, n, out=(r.clone(), t, n.clone(), _ints([0])))
    with pytest.raises(TypeError, match="tuple of 4"):
        tg.kv_fork(cache, r, t, n, out=(r.clone(),))
    with pytest.raises(tg.TgError, match="overlaps"):
        tg.kv_compact(cache, r, t, out=(r.clone(), t, r.clone(), _ints([0])))
    with pytest.raises(ValueError, match="table"):
        tg.kv_compact(cache, r, t[0])
    with pytest.raises(ValueError, match="same heads"):
        tg.kv_copy(cache, _ints([0]), _ints([0]), to=_cache(tg, 4, kv=1))
    with pytest.raises(ValueError, match="dst must have shape"):
        tg.kv_copy(cache, _ints([0]), _ints([0, 1]))
    with pytest.raises(tg.TgError, match="overlap"):
        tg.kv_copy(cache, _ints([0]), _ints([0]), to=tg.KvCache(cache.k[1:], cache.v[1:], cache.k_scale[1:], cache.v_scale[1:]))
    with pytest.raises(TypeError, match="KvCache"):
        tg.kv_copy(cache, _ints([0]), _ints([0]), to=tg.KvCache)
    _status(tg)
