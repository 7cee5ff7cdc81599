"""GPU checks of attention over the paged 8-bit cache against its definition in float64
(tests/kv_reference.py, where the tolerances are derived)."""
import math

import pytest
import torch

from tests import kv_reference as ref

pytestmark = pytest.mark.gpu

HALF = [torch.float16, torch.bfloat16]
CODES = [torch.float8_e4m3fn, torch.int8]


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


def _case(tg, counts, lens, page, kv, share, dim, ct, dt, seed=0, garbage=True):
    """A cache whose used tokens are ordinary and whose unused places (past a sequence's end, unused pages) hold
    NaN codes (e4m3) or large ones, with scales of NaN on unused pages."""
    dtype = CODES[ct]
    g = torch.Generator().manual_seed(seed)
    pages = sum(-(-n // page) for n in lens) + 2
    order = torch.randperm(pages, generator=g)
    table = torch.full((len(lens), max(1, max(-(-n // page) for n in lens))), -1, dtype=torch.int32)
    if dtype is torch.int8:
        k, v = (torch.randint(-127, 128, (pages, kv, page, dim), generator=g, dtype=torch.int8) for _ in range(2))
        mid = 1 / 73.6
    else:
        k, v = ((torch.randn(pages, kv, page, dim, generator=g) * 110).clamp(-448, 448).to(dtype) for _ in range(2))
        mid = 1 / 110
    ks, vs = (torch.rand(pages, kv, generator=g).mul(6).sub(3).exp2() * mid for _ in range(2))
    ks = ks.clamp(max=2 * mid)
    used, at = torch.zeros(pages, page, dtype=torch.bool), 0
    for i, n in enumerate(lens):
        m = -(-n // page)
        table[i, :m] = order[at:at + m]
        at += m
        for s in range(m):
            used[table[i, s], :min(page, n - s * page)] = True
    if garbage:
        code = 0x7F
        for c in (k, v):
            raw = c.view(torch.uint8)
            raw[(~used)[:, None, :, None].expand_as(raw)] = code
        ks[~used.any(1)] = math.nan
        vs[~used.any(1)] = math.nan
    q = (torch.randn(sum(counts), kv * share, dim, generator=g) * 1.5).to(HALF[dt])
    return tg.KvCache(k.cuda(), v.cuda(), ks.cuda(), vs.cuda()), (k, v, ks, vs), table, q


def _check(out, lse, host, table, q, counts, lens, page, causal, window, scale):
    k, v, ks, vs = host
    row = 0
    for i, (n, t) in enumerate(zip(counts, lens)):
        pages = table[i, :-(-t // page)].long()
        sel = slice(row, row + n)
        o, l, tol, ltol = ref.attention(q[sel].double(), ref.gather(k, ks, pages, t), ref.gather(v, vs, pages, t), t, causal, window, scale)
        half = ref.half_step(out.dtype)
        ref.near(out[sel], o, tol + o.abs() * half + 2.0 ** -25, f"sequence {i}")
        if lse is not None:
            ref.near(lse[sel], l, ltol, f"lse of sequence {i}")
        row += n


def _status_ok(tg):
    st, where = tg.tg_device_status(None)
    assert st == tg.OK, f"device status {st} at {where}"


CASES = [  # counts, lens, page, kv heads, query heads a kv head, dim, cache type, element type, causal, window
    ([1], [1], 16, 1, 1, 64, 0, 0, True, 0),
    ([1], [0], 16, 1, 1, 128, 0, 0, True, 0),
    ([1, 1, 1, 1], [5, 0, 16, 17], 16, 2, 4, 128, 0, 0, True, 0),
    ([1] * 6, [63, 64, 65, 1, 300, 0], 64, 8, 4, 128, 0, 1, True, 0),
    ([1] * 3, [1000, 31, 2500], 32, 2, 8, 64, 1, 0, True, 0),
    ([1] * 3, [129, 4000, 127], 128, 1, 7, 128, 1, 1, True, 0),
    ([1] * 2, [700, 90], 64, 3, 5, 64, 0, 0, True, 100),
    ([1] * 2, [700, 90], 16, 2, 16, 128, 0, 1, True, 17),
    ([1], [333], 16, 1, 33, 64, 1, 0, True, 0),
    ([3, 0, 5, 1], [3, 40, 50, 7], 16, 4, 7, 64, 0, 1, True, 0),
    ([5, 2], [200, 129], 64, 2, 3, 128, 1, 0, True, 64),
    ([8, 16, 2], [8, 500, 2], 32, 1, 8, 128, 0, 0, True, 0),
    ([5, 9], [3, 9], 16, 2, 2, 64, 0, 0, True, 0),          # more new rows than tokens: the first see nothing
    ([4, 4], [100, 60], 64, 2, 4, 128, 0, 0, False, 0),
    ([40, 1], [40, 170], 64, 2, 4, 128, 0, 0, True, 0),
    ([130, 33], [300, 33], 32, 1, 8, 64, 1, 1, True, 0),
    ([128], [128], 128, 2, 1, 128, 0, 0, True, 0),
    ([257], [600], 16, 1, 4, 128, 0, 1, True, 0),
    ([200, 77], [900, 450], 128, 2, 3, 128, 1, 0, True, 150),
    ([70, 20], [350, 20], 64, 1, 5, 64, 0, 0, False, 0),
    ([300], [290], 64, 1, 2, 128, 0, 0, True, 0),
    ([64, 129, 1], [1030, 129, 513], 64, 2, 8, 128, 0, 0, True, 0),
    ([300, 140], [1100, 700], 16, 1, 8, 64, 1, 1, True, 333),
    ([90, 0, 200], [90, 5, 0], 32, 2, 16, 128, 1, 1, True, 0),
]


@pytest.mark.parametrize("counts,lens,page,kv,share,dim,ct,dt,causal,window", CASES)
def test_against_definition(tg, counts, lens, page, kv, share, dim, ct, dt, causal, window):
    cache, host, table, q = _case(tg, counts, lens, page, kv, share, dim, ct, dt, seed=sum(lens) + dim)
    cu = [0] + torch.tensor(counts).cumsum(0).tolist()
    out, lse = tg.attention_kv(q.cuda(), cache, table.cuda(), _ints(lens), _ints(cu), max_new=max(counts), max_len=max(max(lens), 1), causal=causal,
                               window=window, return_lse=True)
    _check(out, lse, host, table, q, counts, lens, page, causal, window, dim ** -0.5)
    again = tg.attention_kv(q.cuda(), cache, table.cuda(), _ints(lens), _ints(cu), max_new=max(counts), causal=causal, window=window)
    _status_ok(tg)
    if max(lens) == table.shape[1] * page:
        assert torch.equal(out, again), "not the same from run to run"
    else:  # another bound on the lengths may split the work another way
        _check(again, None, host, table, q, counts, lens, page, causal, window, dim ** -0.5)


@pytest.mark.parametrize("most", [1, 2, 20])
def test_many_sequences_and_run_to_run(tg, most):
    """Ragged lengths, more sequences than SMs, idle slots among them; the same bits every time."""
    g = torch.Generator().manual_seed(most)
    B = 200
    lens = [0 if i % 9 == 4 else int(n) for i, n in enumerate(torch.randint(1, 700, (B,), generator=g))]
    counts = [1 if n < most else most for n in lens]
    cache, host, table, q = _case(tg, counts, lens, 32, 2, 4, 64, 0, 0, seed=21)
    cu = [0] + torch.tensor(counts).cumsum(0).tolist()
    args = (q.cuda(), cache, table.cuda(), _ints(lens), _ints(cu))
    out, lse = tg.attention_kv(*args, max_new=most, max_len=700, return_lse=True)
    _check(out, lse, host, table, q, counts, lens, 32, True, 0, 0.125)
    for _ in range(3):
        again, lagain = tg.attention_kv(*args, max_new=most, max_len=700, return_lse=True)
        assert torch.equal(out, again) and torch.equal(lse, lagain)
    _status_ok(tg)


@pytest.mark.parametrize("counts,lens,dt", [([1], [40000], 0), ([1, 3], [100, 30011], 1), ([9], [20000], 0), ([50, 3], [20000, 300], 0)])
def test_long(tg, counts, lens, dt):
    cache, host, table, q = _case(tg, counts, lens, 64, 2, 4, 128, 0, dt, seed=22)
    cu = [0] + torch.tensor(counts).cumsum(0).tolist()
    out, lse = tg.attention_kv(q.cuda(), cache, table.cuda(), _ints(lens), _ints(cu), max_new=max(counts), max_len=max(lens), return_lse=True)
    _check(out, lse, host, table, q, counts, lens, 64, True, 0, 128 ** -0.5)
    _status_ok(tg)


@pytest.mark.parametrize("counts,lens", [([1, 1], [300, 47]), ([60, 5], [300, 47])])
def test_scales_far_apart(tg, counts, lens):
    """Pages whose value scales are up to 2^40 apart, a page of zeros (scale 2^-60), one large score among small ones."""
    cache, host, table, q = _case(tg, counts, lens, 16, 1, 4, 64, 1, 0, seed=23, garbage=False)
    k, v, ks, vs = host
    pages = table[0, :-(-lens[0] // 16)].long()
    vs[pages] *= torch.logspace(-20, 20, len(pages), base=2.0)[:, None]
    vs[pages[3]] = 2.0 ** -60
    v[pages[3]] = 0
    ks[pages[5]] *= 8
    cache = tg.KvCache(*(t.cuda() for t in host))
    cu = _ints([0] + torch.tensor(counts).cumsum(0).tolist())
    out, lse = tg.attention_kv(q.bfloat16().cuda(), cache, table.cuda(), _ints(lens), cu, max_new=max(counts), max_len=300, return_lse=True)
    _check(out, lse, host, table, q.bfloat16(), counts, lens, 16, True, 0, 0.125)
    _status_ok(tg)


@pytest.mark.parametrize("counts,lens", [([1, 1], [100, 30]), ([50, 30], [100, 30])])
def test_queries_of_every_size(tg, counts, lens):
    """bf16 queries of 2^60 and of 2^-60 (with a scale to match), zero ones, and one row with a NaN."""
    for size in (60, -60):
        cache, host, table, q = _case(tg, counts, lens, 32, 2, 3, 128, 0, 1, seed=24, garbage=False)
        q = (q.float() * 2.0 ** size).bfloat16()
        q[0, 1] = 0
        cu = _ints([0] + torch.tensor(counts).cumsum(0).tolist())
        out, lse = tg.attention_kv(q.cuda(), cache, table.cuda(), _ints(lens), cu, max_new=max(counts), max_len=100, scale=128 ** -0.5 * 2.0 ** -size, return_lse=True)
        _check(out, lse, host, table, q, counts, lens, 32, True, 0, 128 ** -0.5 * 2.0 ** -size)
    q[0, 2, 5] = math.nan
    out = tg.attention_kv(q.cuda(), cache, table.cuda(), _ints(lens), cu, max_new=max(counts), max_len=100)
    assert out[0, 2].isnan().all() and not out[0, [0, 1, 3, 4, 5]].isnan().any() and not out[1:].isnan().any()
    _status_ok(tg)


@pytest.mark.parametrize("most", [4, 30])
def test_nan_in_the_cache_reaches_the_rows_that_see_it_and_no_other_sequence(tg, most):
    counts, lens = [most, 1, most], [40, 33, 35]
    cache, host, table, q = _case(tg, counts, lens, 16, 1, 2, 64, 0, 0, seed=25, garbage=False)
    raw = cache.v.view(torch.uint8)
    raw[int(table[0, 2]), 0, 6, 7] = 0x7F  # sequence 0, position 38: its last two rows see it
    cu = _ints([0, most, most + 1, 2 * most + 1])
    out = tg.attention_kv(q.cuda(), cache, table.cuda(), _ints(lens), cu, max_new=most, max_len=40)
    nan = out.isnan()
    assert nan[most - 2:most, :, 7].all() and not nan[most:].any()
    assert not nan[:, :, :7].any() and not nan[:, :, 8:].any()


@pytest.mark.parametrize("most", [1, 40])
def test_strided_and_unaligned_queries(tg, most):
    counts, lens = [most, 1], [most + 50, 70]
    cache, host, table, q = _case(tg, counts, lens, 64, 2, 4, 128, 0, 0, seed=26)
    cu = _ints([0, most, most + 1])
    T = most + 1
    for off, width in ((0, 16), (1, 16), (8, 9)):
        base = torch.zeros(T * width * 128 + off, dtype=torch.float16, device="cuda")
        x = base[off:].view(T, width, 128)[:, :8]
        x.copy_(q)
        out = tg.attention_kv(x, cache, table.cuda(), _ints(lens), cu, max_new=most, max_len=max(lens))
        _check(out, None, host, table, q, counts, lens, 64, True, 0, 128 ** -0.5)
    x = q.cuda().transpose(0, 1).contiguous().transpose(0, 1)  # heads first in memory
    out = tg.attention_kv(x, cache, table.cuda(), _ints(lens), cu, max_new=most, max_len=max(lens))
    _check(out, None, host, table, q, counts, lens, 64, True, 0, 128 ** -0.5)
    _status_ok(tg)


def test_without_offsets_and_given_output(tg):
    lens = [10, 0, 77]
    cache, host, table, q = _case(tg, [1, 1, 1], lens, 16, 2, 2, 64, 1, 1, seed=27)
    out = torch.full((3, 4, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    assert tg.attention_kv(q.cuda(), cache, table.cuda(), _ints(lens), max_len=80, out=out) is out
    _check(out, None, host, table, q, [1, 1, 1], lens, 16, True, 0, 0.125)


@pytest.mark.parametrize("most", [1, 30])
def test_ranges_are_reported_and_not_followed(tg, most):
    """Page numbers out of range leave their keys out; lengths and offsets out of range leave the sequence's rows
    zero; others are served."""
    counts, lens = [most, most], [64, 100]
    cache, host, table, q = _case(tg, counts, lens, 16, 1, 2, 64, 0, 0, seed=28)
    cu = [0, most, 2 * most]
    good = tg.attention_kv(q.cuda(), cache, table.cuda(), _ints(lens), _ints(cu), max_new=most, max_len=112)
    _status_ok(tg)
    for entry in (-1, 9 + 4, 2 ** 31 - 1, -2 ** 31):
        t = table.clone()
        t[1, 2] = entry
        out = tg.attention_kv(q.cuda(), cache, t.cuda(), _ints(lens), _ints(cu), max_new=most, max_len=112)
        assert tg.tg_device_status(None)[0] == tg.ERR_BOUNDS
        assert torch.equal(out[:most], good[:most]) and out.isfinite().all()
        hidden = [i for i in range(7) if i != 2]
        if most == 1:  # one new row: the keys of the other pages, all visible
            k, v = (torch.cat([ref.gather(c, s, table[1, [i]].long(), 16 if i < 6 else 4) for i in hidden]) for c, s in ((host[0], host[2]), (host[1], host[3])))
            o, _, tol, _ = ref.attention(q[1:].double(), k, v, 84, False, 0, 0.125)
            ref.near(out[1:], o, tol + o.abs() * 2.0 ** -11 + 2.0 ** -25)
    for bad_lens in ([64, 113], [64, -1]):
        out = tg.attention_kv(q.cuda(), cache, table.cuda(), _ints(bad_lens), _ints(cu), max_new=most, max_len=112)
        assert tg.tg_device_status(None)[0] == tg.ERR_BOUNDS
        ref.near(out[:most], good[:most].double().cpu(), 2.0 ** -10 * good[:most].double().abs().cpu() + 2.0 ** -10)
        assert (out[most:] == 0).all()
    out = tg.attention_kv(q.cuda(), cache, table.cuda(), _ints(lens), _ints([0, most, 2 * most + 1]), max_new=most + 1, max_len=112,
                          out=torch.zeros_like(good))
    assert tg.tg_device_status(None)[0] == tg.ERR_BOUNDS
    ref.near(out[:most], good[:most].double().cpu(), 2.0 ** -10 * good[:most].double().abs().cpu() + 2.0 ** -10)
    assert (out[most:] == 0).all()
    _status_ok(tg)


def test_past_four_gigabytes(tg):
    """A page whose codes begin past 2^32 bytes, in a table with one that does not."""
    page, kv, dim = 128, 8, 128
    pages = (1 << 32) // (page * kv * dim) + 8
    for counts in ([1], [70]):
        cache, host, table, q = _case(tg, counts, [200], page, kv, 2, dim, 1, 0, seed=29, garbage=False)
        k = torch.empty(pages, kv, page, dim, dtype=torch.int8, device="cuda")
        v = torch.empty_like(k)
        ks, vs = torch.empty(pages, kv, device="cuda"), torch.empty(pages, kv, device="cuda")
        where = [pages - 1, 0]
        for i in range(2):
            for big, small in ((k, cache.k), (v, cache.v), (ks, cache.k_scale), (vs, cache.v_scale)):
                big[where[i]] = small[int(table[0, i])]
        out = tg.attention_kv(q.cuda(), tg.KvCache(k, v, ks, vs), _ints([where]), _ints([200]), _ints([0, counts[0]]), max_new=counts[0], max_len=200)
        _check(out, None, host, table, q, counts, [200], page, True, 0, 128 ** -0.5)
    _status_ok(tg)


@pytest.mark.parametrize("most", [1, 24])
def test_other_stream_and_graph(tg, most):
    counts, lens = [most, most], [500, 90]
    cache, host, table, q = _case(tg, counts, lens, 16, 2, 4, 64, 0, 0, seed=30)
    table_d, cu = table.cuda(), _ints([0, most, 2 * most])
    dev, lens_d = torch.zeros_like(q).cuda(), _ints([1, 0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        tg.attention_kv(dev, cache, table_d, lens_d, cu, max_new=most, max_len=512)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = tg.attention_kv(dev, cache, table_d, lens_d, cu, max_new=most, max_len=512)
    dev.copy_(q)
    lens_d.copy_(_ints(lens))
    graph.replay()
    torch.cuda.synchronize()
    _check(out, None, host, table, q, counts, lens, 16, True, 0, 0.125)
    side.wait_stream(torch.cuda.current_stream())
    other = tg.attention_kv(dev, cache, table_d, lens_d, cu, max_new=most, max_len=512, stream=side)
    side.synchronize()
    assert torch.equal(other, out)
    _status_ok(tg)
