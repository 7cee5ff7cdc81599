"""CPU checks of the entry points around pages, shared prefixes and drawing: refusals on the host, before anything
touches a device, and the sizes of their workspaces."""
import math

import pytest

K, V, KS, VS = 0x10000000, 0x20000000, 0x30000000, 0x31000000
TK, TV, TKS, TVS = 0x40000000, 0x50000000, 0x60000000, 0x61000000
REFS, TABLE, LENS, PARENTS, GROUPS, SHARED, CU = (0x70000000 + i * 0x100000 for i in range(7))
REFS_OUT, TABLE_OUT, LENS_OUT, SPARE, MOVED, TOKENS = (0x78000000 + i * 0x100000 for i in range(6))
WORK, Q, O, U = 0x80000000, 0x90000000, 0xA0000000, 0xB0000000
POINTERS = ("k", "v", "ks", "vs", "tk", "tv", "tks", "tvs", "src", "dst", "refs", "table", "lens", "parents", "refs_out", "table_out", "lens_out", "spare", "moved", "used",
            "work", "q", "o", "groups", "shared", "cu", "x", "u", "t", "tk_", "tp", "tm", "tokens")


@pytest.fixture(scope="module")
def tg():
    import __graft_entry__
    __graft_entry__.build()
    import tiled_tensor_core_tcgen05_gb300 as m
    return m


def _args(defaults, changes):
    d = dict(defaults)
    for key, x in changes.items():
        assert key in d, key
        d[key] = x
    return [None if x == 0 and key in POINTERS else x for key, x in d.items()]


CACHE = dict(k=K, v=V, ks=KS, vs=VS, pages=100, kv_heads=8, page=64, dim=128, fmt=0)
COPY = dict(k=K, v=V, ks=KS, vs=VS, pages=100, tk=TK, tv=TV, tks=TKS, tvs=TVS, to_pages=100, kv_heads=8, page=64, dim=128, fmt=0, src=REFS, dst=TABLE, count=5, stream=None)
FORK = dict(CACHE, refs=REFS, table=TABLE, width=16, lens=LENS, batch=4, parents=PARENTS, count=7, room=1, refs_out=REFS_OUT, table_out=TABLE_OUT, lens_out=LENS_OUT, spare=SPARE,
            work=WORK, work_bytes=1 << 20, stream=None)
COMPACT = dict(CACHE, refs=REFS, table=TABLE, width=16, batch=4, refs_out=REFS_OUT, table_out=TABLE_OUT, moved=MOVED, used=SPARE, work=WORK, work_bytes=1 << 20, stream=None)
SHARE = dict(q=Q, qt=4096, qh=128, o=O, lse=None, **CACHE, table=TABLE, width=16, lens=LENS, cu=CU, batch=4, total=7, heads=32, max_new=3, max_len=1024, causal=1, groups=GROUPS,
             shared=SHARED, group_count=2, max_rows=7, scale=0.1, dtype=0, work=WORK, work_bytes=1 << 20, stream=None)
SAMPLE = dict(x=Q, stride=1000, rows=4, vocab=1000, dtype=0, u=U, t=0, t_all=1.0, tk_=0, k_all=0, tp=0, p_all=1.0, tm=0, m_all=0.0, tokens=TOKENS, stream=None)


@pytest.mark.parametrize("call,defaults,changes,says", [
    ("tg_kv_copy", COPY, dict(page=48), "page must be"),
    ("tg_kv_copy", COPY, dict(dim=96), "head dimensions"),
    ("tg_kv_copy", COPY, dict(fmt=2), "format"),
    ("tg_kv_copy", COPY, dict(count=-1), "count"),
    ("tg_kv_copy", COPY, dict(src=0), "NULL"),
    ("tg_kv_copy", COPY, dict(dst=TABLE + 2), "aligned"),
    ("tg_kv_copy", COPY, dict(tv=0), "NULL"),
    ("tg_kv_copy", COPY, dict(tk=TK + 8), "16-byte"),
    ("tg_kv_copy", COPY, dict(tk=K), "overlap"),
    ("tg_kv_copy", COPY, dict(tk=K, tv=V, tks=KS, tvs=VS, to_pages=99), "overlap"),
    ("tg_kv_copy", COPY, dict(src=TV + 64), "overlap"),
    ("tg_kv_copy", COPY, dict(pages=1 << 30), "too large"),
    ("tg_kv_fork", FORK, dict(room=-1), "room"),
    ("tg_kv_fork", FORK, dict(room=1 << 31), "room"),
    ("tg_kv_fork", FORK, dict(batch=-1), "out of range"),
    ("tg_kv_fork", FORK, dict(count=(1 << 20) + 1), "out of range"),
    ("tg_kv_fork", FORK, dict(width=1 << 30), "out of range"),
    ("tg_kv_fork", FORK, dict(parents=0), "without parents"),
    ("tg_kv_fork", FORK, dict(lens=0), "NULL"),
    ("tg_kv_fork", FORK, dict(refs=0), "NULL"),
    ("tg_kv_fork", FORK, dict(spare=0), "NULL"),
    ("tg_kv_fork", FORK, dict(table_out=TABLE_OUT + 1), "aligned"),
    ("tg_kv_fork", FORK, dict(work=0), "workspace"),
    ("tg_kv_fork", FORK, dict(work_bytes=100), "workspace of"),
    ("tg_kv_fork", FORK, dict(work=WORK + 8), "16-byte"),
    ("tg_kv_fork", FORK, dict(refs_out=REFS + 4), "overlaps"),
    ("tg_kv_fork", FORK, dict(table_out=TABLE), "overlaps"),
    ("tg_kv_fork", FORK, dict(lens_out=LENS), "overlaps"),
    ("tg_kv_fork", FORK, dict(spare=LENS_OUT + 24), "overlaps"),
    ("tg_kv_fork", FORK, dict(parents=K + 256), "overlaps"),
    ("tg_kv_compact", COMPACT, dict(moved=0), "NULL"),
    ("tg_kv_compact", COMPACT, dict(used=0), "NULL"),
    ("tg_kv_compact", COMPACT, dict(batch=-3), "out of range"),
    ("tg_kv_compact", COMPACT, dict(work_bytes=8), "workspace of"),
    ("tg_kv_compact", COMPACT, dict(table_out=TABLE + 8), "overlaps"),
    ("tg_kv_compact", COMPACT, dict(moved=REFS_OUT + 40), "overlaps"),
    ("tg_attention_kv_shared", SHARE, dict(group_count=-1), "groups"),
    ("tg_attention_kv_shared", SHARE, dict(group_count=5), "as many groups"),
    ("tg_attention_kv_shared", SHARE, dict(max_rows=0), "max_rows"),
    ("tg_attention_kv_shared", SHARE, dict(groups=0), "NULL"),
    ("tg_attention_kv_shared", SHARE, dict(shared=SHARED + 2), "aligned"),
    ("tg_attention_kv_shared", SHARE, dict(causal=2), "causal"),
    ("tg_attention_kv_shared", SHARE, dict(heads=30), "multiple"),
    ("tg_attention_kv_shared", SHARE, dict(scale=math.inf), "scale"),
    ("tg_attention_kv_shared", SHARE, dict(o=Q), "overlaps"),
    ("tg_attention_kv_shared", SHARE, dict(q=0), "NULL"),
])
def test_refusals(tg, call, defaults, changes, says):
    with pytest.raises(tg.TgError) as e:
        getattr(tg, call)(*_args(defaults, changes))
    assert e.value.status == tg.ERR_INVALID_ARG and says in str(e.value), str(e.value)


@pytest.mark.parametrize("changes,says", [
    (dict(dtype=3), "dtype"), (dict(rows=-1), "sizes"), (dict(rows=(1 << 24) + 1), "sizes"), (dict(vocab=(1 << 18) + 1), "vocab"), (dict(vocab=0), "nothing to draw"),
    (dict(stride=-1), "row_stride"), (dict(stride=1 << 31), "row_stride"), (dict(t_all=math.nan), "numbers"), (dict(p_all=math.nan), "numbers"), (dict(m_all=math.nan), "numbers"),
    (dict(x=0), "NULL"), (dict(u=0), "NULL"), (dict(tokens=0), "NULL"), (dict(x=Q + 1), "aligned to its type"), (dict(dtype=2, x=Q + 2), "aligned to its type"),
    (dict(u=U + 1), "4-byte"), (dict(tm=U + 3), "4-byte"), (dict(tokens=Q + 16), "overlaps"), (dict(tokens=U), "overlaps"), (dict(t=TOKENS), "overlaps"),
])
def test_sample_refusals(tg, changes, says):
    with pytest.raises(tg.TgError) as e:
        tg.tg_sample(*_args(SAMPLE, changes))
    assert e.value.status == tg.ERR_INVALID_ARG and says in str(e.value), str(e.value)


def test_calls_of_nothing_need_no_device(tg):
    tg.tg_kv_copy(*_args(COPY, dict(count=0, src=0, dst=0)))
    tg.tg_sample(*_args(SAMPLE, dict(rows=0, x=0, u=0, tokens=0)))
    tg.tg_attention_kv_shared(*_args(SHARE, dict(total=0, batch=0, group_count=0, groups=0, shared=0, q=0, o=0, cu=0, work=0)))


def test_workspaces(tg):
    assert tg.tg_kv_compact_workspace(0) > 0 and tg.tg_kv_compact_workspace(1000) >= 500 * 12
    one, two = tg.tg_kv_fork_workspace(100, 64, 4, 4, 16), tg.tg_kv_fork_workspace(100000, 64, 400, 500, 16)
    assert 0 < one < two and two >= 500 * (12 + 4 + 8) + 400 * 20 + 8000 * 4
    for call, args in ((tg.tg_kv_fork_workspace, (10, 48, 1, 1, 1)), (tg.tg_kv_fork_workspace, (-1, 64, 1, 1, 1)), (tg.tg_kv_fork_workspace, (10, 64, 1, -1, 1)), (tg.tg_kv_compact_workspace, (-1,))):
        with pytest.raises(tg.TgError):
            call(*args)
