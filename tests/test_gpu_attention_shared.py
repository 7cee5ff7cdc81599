"""GPU checks of attention over a prefix that sequences share, against the definition in float64 over each sequence's
own table (tests/kv_reference.py). Beyond the tolerances derived there, the two passes' results are added with two powers
of two good to 2^-21 each: 2^-19 of the largest value covers them."""
import pytest
import torch

from tests import kv_reference as ref
from tests import test_gpu_attention_kv as attend

pytestmark = pytest.mark.gpu
_ints, _status_ok = attend._ints, attend._status_ok


@pytest.fixture(scope="module")
def tg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import tiled_tensor_core_tcgen05_gb300 as m
    torch.cuda.set_device(0)
    return m


@pytest.fixture(autouse=True)
def always(tg):
    """The sizes here would not pay a pass of their own."""
    tg.tg_debug_share_always(True)
    yield
    tg.tg_debug_share_always(False)


def _share(table, groups, shared, lens, page):
    """Makes the sequences of each group begin with the pages of the group's longest."""
    for g, n in enumerate(shared):
        members = range(groups[g], groups[g + 1])
        if not members:
            continue
        whole = max(members, key=lambda i: lens[i])
        m = -(-n // page)
        for i in members:
            if lens[i] >= n:
                table[i, :m] = table[whole, :m]


def _check(out, lse, host, table, q, counts, lens, page, causal, scale):
    k, v, ks, vs = host
    row = 0
    for i, (n, t) in enumerate(zip(counts, lens)):
        pages = table[i, :-(-t // page)].long()
        sel = slice(row, row + n)
        values = ref.gather(v, vs, pages, t)
        o, l, tol, ltol = ref.attention(q[sel].double(), ref.gather(k, ks, pages, t), values, t, causal, 0, scale)
        half = ref.half_step(out.dtype)
        more = 2.0 ** -19 * values.abs().max() if t else 0.0
        ref.near(out[sel], o, tol + more + o.abs() * half + 2.0 ** -25, f"sequence {i}")
        if lse is not None:
            ref.near(lse[sel], l, ltol + 2.0 ** -19, f"lse of sequence {i}")
        row += n


CASES = [  # groups, shared, counts, lens, page, kv heads, query heads a kv head, dim, cache type, element type, causal
    ([0, 1], [0], [1], [5], 16, 1, 1, 64, 0, 0, True),
    ([0, 1], [64], [1], [65], 16, 1, 1, 128, 0, 0, True),
    ([0, 4], [640], [1] * 4, [641, 700, 1300, 650], 64, 2, 4, 128, 0, 0, True),
    ([0, 4], [600], [1] * 4, [700, 641, 1300, 650], 64, 2, 4, 128, 0, 1, True),        # no whole number of pages
    ([0, 3, 3, 8], [128, 64, 320], [1] * 8, [129, 400, 128, 0, 321, 700, 320, 322], 16, 2, 4, 64, 1, 0, True),  # an empty group, idle and short sequences
    ([1, 3], [256], [1] * 5, [300, 300, 299, 17, 500], 32, 3, 5, 64, 0, 1, True),      # sequences in no group on both sides
    ([0, 5], [1024], [3, 1, 5, 2, 4], [1100, 1025, 1029, 2000, 1028], 128, 1, 7, 128, 1, 1, True),
    ([0, 70], [512], [1] * 70, [513 + 3 * i for i in range(70)], 64, 1, 4, 128, 0, 0, True),   # the first pass on tcgen05
    ([0, 40, 41, 100], [1000, 320, 64], [1 + i % 3 for i in range(100)], [1003 + i for i in range(100)], 16, 2, 7, 64, 1, 1, True),
    ([0, 6], [200], [2] * 6, [202, 203, 300, 201, 64, 900], 16, 2, 2, 64, 0, 0, False),
    ([0, 2], [64], [30, 12], [100, 90], 16, 2, 4, 64, 0, 0, True),                     # many rows a sequence: as without groups
    ([0, 2], [1024], [1, 1], [1025, 1090], 128, 1, 64, 128, 0, 1, True),
    ([0, 3], [20032], [1, 2, 1], [20100, 20034, 30000], 64, 1, 2, 64, 0, 0, True),     # few groups, long
]


@pytest.mark.parametrize("groups,shared,counts,lens,page,kv,share,dim,ct,dt,causal", CASES)
def test_against_definition(tg, groups, shared, counts, lens, page, kv, share, dim, ct, dt, causal):
    cache, host, table, q = attend._case(tg, counts, lens, page, kv, share, dim, ct, dt, seed=sum(lens) + dim)
    _share(table, groups, shared, lens, page)
    cu = [0] + torch.tensor(counts).cumsum(0).tolist()
    args = (q.cuda(), cache, table.cuda(), _ints(lens), _ints(groups), _ints(shared), _ints(cu))
    rows = max(cu[b] - cu[a] for a, b in zip(groups, groups[1:]))
    how = dict(max_new=max(counts), max_len=max(lens), causal=causal, return_lse=True)
    out, lse = tg.attention_kv_shared(*args, max_rows=rows, **how)
    _status_ok(tg)
    _check(out, lse, host, table, q, counts, lens, page, causal, dim ** -0.5)
    again, lagain = tg.attention_kv_shared(*args, max_rows=rows, **how)
    assert torch.equal(out, again) and torch.equal(lse, lagain), "not the same from run to run"
    loose = tg.attention_kv_shared(*args, max_new=max(counts), causal=causal)  # bounds left to the call
    _check(loose, None, host, table, q, counts, lens, page, causal, dim ** -0.5)
    if max(counts) == 1:
        _check(tg.attention_kv_shared(*args[:-1], **how)[0], None, host, table, q, counts, lens, page, causal, dim ** -0.5)
    _status_ok(tg)


def test_groups_out_of_range(tg):
    """Reported, and the sequences attended by themselves."""
    counts, lens, page = [1] * 6, [200, 210, 230, 300, 190, 260], 16
    cache, host, table, q = attend._case(tg, counts, lens, page, 2, 4, 64, 0, 0)
    _share(table, [0, 6], [128], lens, page)
    run = lambda groups, shared, **how: tg.attention_kv_shared(q.cuda(), cache, table.cuda(), _ints(lens), _ints(groups), _ints(shared), **how)  # noqa: E731
    for groups, shared, how in (([0, 7], [128], {}), ([-1, 6], [128], {}), ([4, 2], [128], {}), ([0, 5, 3, 6], [128] * 3, {}), ([0, 6], [-1], {}), ([0, 6], [100000], {}),
                                ([0, 6], [128], dict(max_rows=5)), ([0, 3, 6], [128, -5], {}), ([0, 6], [301], dict(max_len=300))):
        out = run(groups, shared, **how)
        st, _ = tg.tg_device_status(None)
        assert st == tg.ERR_BOUNDS, (groups, shared, how)
        _check(out, None, host, table, q, counts, lens, page, True, 0.125)
    _check(run([0], []), None, host, table, q, counts, lens, page, True, 0.125)  # no groups
    _status_ok(tg)


def test_lengths_and_offsets_out_of_range(tg):
    """What tg_attention_kv does with them, beside a group that is in order."""
    counts, lens, page = [1] * 6, [200, 210, 230, 300, 190, 260], 16
    cache, host, table, q = attend._case(tg, counts, lens, page, 2, 4, 64, 0, 0)
    _share(table, [0, 6], [128], lens, page)
    bad = [200, -4, 230, 100000, 190, 260]
    out, lse = tg.attention_kv_shared(q.cuda(), cache, table.cuda(), _ints(bad), _ints([0, 6]), _ints([128]), return_lse=True)
    assert tg.tg_device_status(None)[0] == tg.ERR_BOUNDS
    good = [n if 0 <= n <= 304 else 0 for n in bad]
    _check(out, lse, host, table, q, counts, good, page, True, 0.125)
    out = tg.attention_kv_shared(q.cuda(), cache, table.cuda(), _ints(lens), _ints([1, 6]), _ints([128]), _ints([0, 1, 2, 3, 4, 5, 5]))  # a row of no sequence
    assert (out[5] == 0).all()
    _check(out[:5], None, host, table, q, counts[:5], lens[:5], page, True, 0.125)
    _status_ok(tg)
    table[2, 3] = 10 ** 6  # a page the group does not read: its first sequence's are the ones that count
    out = tg.attention_kv_shared(q.cuda(), cache, table.cuda(), _ints(lens), _ints([0, 6]), _ints([128]))
    table[2, 3] = table[0, 3]
    _check(out, None, host, table, q, counts, lens, page, True, 0.125)
    _status_ok(tg)


def test_what_a_nan_in_the_prefix_reaches(tg):
    counts, lens, page = [1] * 5, [200, 210, 230, 300, 190], 16
    cache, host, table, q = attend._case(tg, counts, lens, page, 2, 4, 64, 0, 0)
    _share(table, [0, 3], [128], lens, page)
    cache.v.view(torch.uint8)[table[0, 1], 0, 3] = 0x7F
    out = tg.attention_kv_shared(q.cuda(), cache, table.cuda(), _ints(lens), _ints([0, 3]), _ints([128]))
    assert out[:3, :4].isnan().all() and out[3:].isfinite().all() and out[:3, 4:].isfinite().all()
    _status_ok(tg)


@pytest.mark.parametrize("n,length", [(3, 700), (70, 8200)])  # too little to share, and enough
def test_what_the_call_chooses(tg, n, length):
    tg.tg_debug_share_always(False)
    counts, lens, page = [1] * n, [length - 3 * (i % 5) for i in range(n)], 64
    cache, host, table, q = attend._case(tg, counts, lens, page, 2, 8, 128, 0, 0)
    _share(table, [0, n], [640], lens, page)
    out, lse = tg.attention_kv_shared(q.cuda(), cache, table.cuda(), _ints(lens), _ints([0, n]), _ints([640]), max_len=length, return_lse=True)
    _check(out, lse, host, table, q, counts, lens, page, True, 128 ** -0.5)
    _status_ok(tg)


def test_strides_streams_graphs_and_out(tg):
    counts, lens, page = [1] * 12, [400 + 17 * i for i in range(12)], 32
    cache, host, table, q = attend._case(tg, counts, lens, page, 2, 4, 128, 1, 1)
    _share(table, [0, 12], [384], lens, page)
    args = [table.cuda(), _ints(lens), _ints([0, 12]), _ints([384])]
    wide = torch.randn(12, 12, 128, dtype=q.dtype, device="cuda")
    wide[:, 2:10] = q.cuda()
    want = tg.attention_kv_shared(q.cuda(), cache, *args)
    out = torch.empty_like(want)
    assert tg.attention_kv_shared(wide[:, 2:10], cache, *args, out=out) is out and torch.equal(out, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = tg.attention_kv_shared(q.cuda(), cache, *args, stream=side)
    side.synchronize()
    assert torch.equal(other, want)
    dq, lengths = q.cuda(), args[1]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = tg.attention_kv_shared(dq, cache, *args)
    lens[3], lens[7] = 300, 385  # one is too short now
    lengths.copy_(_ints(lens))
    dq.mul_(0.5)
    graph.replay()
    _check(got, None, host, table, q * 0.5, counts, lens, page, True, 128 ** -0.5)
    _status_ok(tg)


def test_refusals(tg):
    cache, _, table, q = attend._case(tg, [1, 1], [40, 40], 16, 2, 2, 64, 0, 0)
    q, table, lens, groups, shared = q.cuda(), table.cuda(), _ints([40, 40]), _ints([0, 2]), _ints([16])
    with pytest.raises(ValueError, match="groups must have shape"):
        tg.attention_kv_shared(q, cache, table, lens, _ints([0]), shared)
    with pytest.raises(TypeError, match="int32"):
        tg.attention_kv_shared(q, cache, table, lens, groups, shared.long())
    with pytest.raises(ValueError, match="shared must be a vector"):
        tg.attention_kv_shared(q, cache, table, lens, groups, _ints([[16]]))
    with pytest.raises(tg.TgError, match="max_rows"):
        tg.attention_kv_shared(q, cache, table, lens, groups, shared, max_rows=0)
    with pytest.raises(tg.TgError, match="as many groups"):
        tg.attention_kv_shared(q, cache, table, lens, _ints([0, 1, 2, 2]), _ints([1, 1, 1]))
    with pytest.raises(tg.TgError, match="overlaps"):
        tg.attention_kv_shared(q, cache, table, lens, groups, shared, out=q)
    with pytest.raises(ValueError, match="Q must have shape"):
        tg.attention_kv_shared(q[:, :, :32], cache, table, lens, groups, shared)
    _status_ok(tg)
