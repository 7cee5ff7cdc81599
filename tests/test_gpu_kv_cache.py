"""GPU checks of rotary positions, of writing the paged 8-bit cache and of reading it back, against the
definitions in float64 (tests/kv_reference.py). Tolerances: half a rounding step of the result's type, plus
the 32-bit error of the terms."""
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


def _status_ok(tg):
    st, where = tg.tg_device_status(None)
    assert st == tg.OK, f"device status {st} at {where}"


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- rotary positions

def _near_rotated(y, want, size, dtype, what=""):
    # cos and sin are off by at most 2^-22 (their own 2^-23 and the angle), the products and the sum by 2^-24 each
    tol = want.abs() * ref.half_step(dtype) * (1 + 2.0 ** -10) + size * 2.0 ** -21 + 2.0 ** -25
    ref.near(y, want, tol, what)


ROPE = [  # tokens, heads, dim, rotary, interleaved, backward, dtype, first position
    (1, 1, 64, 64, False, False, 0, 0), (1, 40, 128, 128, False, False, 0, 4095), (7, 3, 128, 128, True, False, 1, 1 << 20),
    (33, 5, 64, 32, False, True, 0, 100000), (129, 7, 128, 112, True, True, 1, 2 ** 31 - 200), (5, 2, 64, 48, False, False, 1, 77),
    (3, 2, 80, 2, False, False, 0, 5), (2, 3, 10, 6, True, False, 0, 12345678), (4, 1, 128, 0, False, False, 1, 9), (300, 32, 128, 64, False, False, 0, 0),
    (3, 3, 5, 4, False, False, 0, 3), (2, 2, 256, 256, False, True, 0, 50), (1500, 9, 64, 64, True, False, 0, 31),
]


@pytest.mark.parametrize("T,H,D,rotary,inter,back,dt,first", ROPE)
def test_rope(tg, T, H, D, rotary, inter, back, dt, first):
    dtype = HALF[dt]
    g = torch.Generator().manual_seed(T * 1000 + D)
    x = torch.randn(T, H, D, generator=g).to(dtype)
    pos = torch.arange(first, first + T)
    f = ref.freqs(rotary) if rotary else torch.empty(0, dtype=torch.float64)
    layout = tg.ROPE_INTERLEAVED if inter else tg.ROPE_HALF
    y = tg.rope(x.cuda(), pos.to(torch.int32).cuda(), f.cuda(), 1.25, layout=layout, backward=back)
    assert y.dtype == dtype and y.shape == x.shape
    want, size = ref.rope(x, pos, f, 1.25, inter, back)
    _near_rotated(y, want, size, dtype)
    assert torch.equal(y.cpu()[..., rotary:], x[..., rotary:])
    _status_ok(tg)


@pytest.mark.parametrize("dt", [0, 1])
@pytest.mark.parametrize("off", [0, 1])
def test_rope_slices_in_place_and_negative_positions(tg, dt, off):
    """Heads of a packed projection, rotated where they are (off 1: not 16-byte aligned), the rest untouched."""
    dtype = HALF[dt]
    packed = torch.randn(9, 12 * 64 + 8, generator=torch.Generator().manual_seed(5)).to(dtype)
    dev = packed.cuda()
    x = dev[:, off:off + 6 * 64].view(9, 6, 64)
    pos = torch.tensor([0, -1, 5, 5, -100000, 3, 2 ** 31 - 1, -2 ** 31, 8])
    f = ref.freqs(64)
    assert tg.rope(x, pos.to(torch.int32).cuda(), f.cuda(), out=x) is x
    want, size = ref.rope(packed[:, off:off + 384].view(9, 6, 64), pos, f, 1.0, False)
    _near_rotated(x, want, size, dtype)
    rest = torch.ones(packed.shape[1], dtype=torch.bool)
    rest[off:off + 384] = False
    assert torch.equal(dev.cpu()[:, rest], packed[:, rest])


def test_rope_heads_with_stride_and_transposed_order(tg):
    x = torch.randn(4, 10, 128, generator=torch.Generator().manual_seed(6)).half()
    f, pos = ref.freqs(128), torch.arange(10)
    y = tg.rope(x.cuda().transpose(0, 1), pos.int().cuda(), f.cuda())  # (tokens, heads) stored heads first
    want, size = ref.rope(x.transpose(0, 1), pos, f, 1.0, False)
    _near_rotated(y, want, size, torch.float16)
    y = tg.rope(x.cuda()[:, 1::3], _ints([3, 2, 1, 0]), f.cuda())
    want, size = ref.rope(x[:, 1::3], torch.tensor([3, 2, 1, 0]), f, 1.0, False)
    _near_rotated(y, want, size, torch.float16)


def test_rope_backward_against_differences(tg):
    """sum(dy * rope(x + e)) - sum(dy * rope(x - e)) over 2 e, for one e after another, against the gradient."""
    g = torch.Generator().manual_seed(8)
    dy = torch.randn(2, 1, 8, generator=g).half()
    pos, f = _ints([3, 40000]), ref.freqs(8).cuda()
    dx = tg.rope(dy.cuda(), pos, f, 0.75, backward=True).double().cpu()
    x = torch.zeros(2, 1, 8).half()
    for t in range(2):
        for d in range(8):
            e = torch.zeros_like(x)
            e[t, 0, d] = 1.0
            up, down = (tg.rope(v.cuda(), pos, f, 0.75).double().cpu() for v in (e, -e))
            diff = ((up - down) / 2 * dy.double()).sum()
            # each of the two terms carries the rounding of two rotated values, at most 0.75 each
            assert abs(diff - dx[t, 0, d]) <= 4 * 2.0 ** -11 * 0.75 * dy.double().abs().max() + abs(dx[t, 0, d]) * 2.0 ** -11


# ---------------------------------------------------------------- the cache

def _cache(tg, pages, heads, page, dim, dtype, seed=0, scale=1 / 100):
    g = torch.Generator().manual_seed(seed)
    if dtype is torch.int8:
        k, v = (torch.randint(-127, 128, (pages, heads, page, dim), generator=g, dtype=torch.int8) for _ in range(2))
    else:
        k, v = ((torch.randn(pages, heads, page, dim, generator=g) * 110).clamp(-448, 448).to(dtype) for _ in range(2))
    ks, vs = (torch.rand(pages, heads, generator=g).add(0.1) * scale for _ in range(2))
    return tg.KvCache(k.cuda(), v.cuda(), ks.cuda(), vs.cuda()), (k, v, ks, vs)


def _table(lens, page, pages, seed, width=None):
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    order = torch.randperm(pages, generator=g)
    t = torch.full((len(lens), width or max(1, max(need))), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        t[i, :n] = order[at:at + n]
        at += n
    assert at <= pages
    return t


def _check_codes(got, units, written, before, dtype, slack, what):
    """Every written code is the nearest to its unrounded value (or, within `slack` of half a step, the other), and
    no other changed."""
    raw, old = got.cpu().view(torch.uint8), before.view(torch.uint8)
    assert torch.equal(raw[~written], old[~written]), f"{what}: a code outside the call's tokens changed"
    u = units.clamp(-ref.QMAX[dtype], ref.QMAX[dtype])
    q = got.cpu().double()
    bad = (q - u).abs() > ref.code_step(u, dtype) / 2 + slack * u.abs()
    bad &= written
    assert not bad.any(), f"{what}: {int(bad.sum())} codes are not the nearest"


APPEND = [  # counts, lens, page, heads, dim, cache type, element type, cu given
    ([1], [0], 16, 1, 64, 0, 0, False), ([1, 1, 1], [0, 15, 16], 16, 2, 128, 1, 1, False), ([1] * 9, [0, 1, 62, 63, 64, 65, 127, 128, 300], 64, 8, 128, 0, 1, True),
    ([1] * 5, [0, 127, 128, 200, 1000], 128, 3, 64, 1, 0, False), ([5, 0, 64, 1, 17], [3, 9, 0, 64, 60], 32, 4, 128, 0, 0, True),
    ([130, 1, 257], [0, 5, 63], 64, 2, 64, 1, 1, True), ([16, 32, 48], [0, 16, 8], 16, 5, 64, 0, 1, True), ([300], [77], 128, 8, 128, 1, 0, True),
    ([0, 0, 3], [4, 0, 0], 64, 1, 128, 0, 0, True), ([2, 8, 4], [15, 15, 31], 16, 7, 128, 0, 0, True), ([1000, 513], [0, 100], 32, 2, 128, 1, 0, True),
    ([0, 700, 0, 40, 0], [9, 130, 0, 100, 7], 128, 2, 128, 0, 1, True),
]


@pytest.mark.parametrize("counts,lens,page,heads,dim,ct,dt,given", APPEND)
@pytest.mark.parametrize("rotate", [False, True])
def test_append(tg, counts, lens, page, heads, dim, ct, dt, given, rotate):
    dtype, half = CODES[ct], HALF[dt]
    total = [a + b for a, b in zip(counts, lens)]
    pages = sum(-(-t // page) for t in total) + 3
    cache, before = _cache(tg, pages, heads, page, dim, dtype, seed=page + dim)
    table = _table(total, page, pages, 1)
    g = torch.Generator().manual_seed(2)
    T = sum(counts)
    # rows of very different sizes, so that scales of partly filled pages grow, or stay
    k, v = (torch.randn(T, heads, dim, generator=g) * torch.rand(T, heads, 1, generator=g) for _ in range(2))
    k, v = k.to(half), v.to(half)
    cu = [0] + torch.tensor(counts).cumsum(0).tolist()
    args = (cache, k.cuda(), v.cuda(), table.cuda(), _ints(lens), _ints(cu) if given else None)
    kd, slack = k.double(), 2.0 ** -22
    if rotate:
        q = torch.randn(T, 3 * heads, dim, generator=g).to(half)
        f = ref.freqs(dim)
        pos = torch.cat([torch.arange(a, a + n) for a, n in zip(lens, counts)])
        rq = tg.kv_append(*args, max_new=max(counts), Q=q.cuda(), inv_freq=f.cuda(), amplitude=1.125)
        want, size = ref.rope(q, pos, f, 1.125, False)
        _near_rotated(rq, want, size, half, "queries")
        kd, size = ref.rope(k, pos, f, 1.125, False)
    else:
        assert tg.kv_append(*args, max_new=max(counts)) is None
    for what, x, got, gs, old, olds, rotated in (("keys", kd, cache.k, cache.k_scale, before[0], before[2], rotate),
                                                 ("values", v.double(), cache.v, cache.v_scale, before[1], before[3], False)):
        units, scales, written = ref.append(x, old, olds, table, lens, counts, page, dtype)
        loose = 2.0 ** -20 if rotated else 0  # a rotated value is off by 2^-21 of |a| + |b|, at most 2 of the pair's size
        ref.near(gs, scales, scales * (2.0 ** -23 + loose), what + " scales")
        if rotated:
            units_tol = 2.0 ** -20 * ref.QMAX[dtype]
            u = units.clamp(-ref.QMAX[dtype], ref.QMAX[dtype])
            bad = ((got.cpu().double() - u).abs() > ref.code_step(u, dtype) / 2 + units_tol) & written
            assert not bad.any(), what
            assert torch.equal(got.cpu().view(torch.uint8)[~written], old.view(torch.uint8)[~written])
        else:
            _check_codes(got, units, written, old, dtype, slack, what)
    _status_ok(tg)


@pytest.mark.parametrize("ct", [0, 1])
@pytest.mark.parametrize("most", [1, 40])
def test_append_special_values(tg, ct, most):
    """Zeros, infinities, NaN, the largest and the smallest finite values; the first page starts from garbage."""
    dtype = CODES[ct]
    cache, before = _cache(tg, 8, 1, 32, 64, dtype)
    before[2].fill_(math.nan)
    cache.k_scale.fill_(math.nan)
    T = most
    k = torch.zeros(T, 1, 64)
    v = torch.randn(T, 1, 64, generator=torch.Generator().manual_seed(1))
    v[0, 0, :4] = torch.tensor([math.inf, -math.inf, math.nan, 0.0])
    v[-1, 0, 5:8] = torch.tensor([3.3895e38, -1e-40, 2.0 ** -70])
    v = v.bfloat16()
    table = _table([T], 32, 8, 3)
    tg.kv_append(cache, k.bfloat16().cuda(), v.cuda(), table.cuda(), _ints([0]), _ints([0, T]), max_new=most)
    for p in table[0, :-(-T // 32)].tolist():
        assert cache.k_scale[p, 0].item() == 2.0 ** -60
    n = min(T, 32)
    assert (cache.k.cpu()[int(table[0, 0])].double()[0, :n] == 0).all()
    units, scales, written = ref.append(v.double(), before[1], before[3], table, [0], [T], 32, dtype)
    ref.near(cache.v_scale, scales, scales * 2.0 ** -23)
    got = cache.v.cpu().double()
    if dtype is torch.int8:
        units = units.nan_to_num(nan=0.0)
    assert torch.equal(got.isnan(), units.isnan() & written | before[1].double().isnan())
    u = units.clamp(-ref.QMAX[dtype], ref.QMAX[dtype])
    bad = ((got - u).abs() > ref.code_step(u, dtype) / 2 + 2.0 ** -22 * u.abs()) & written & ~u.isnan()
    assert not bad.any()
    _status_ok(tg)


def test_append_token_by_token_equals_its_definition_over_steps(tg):
    """Forty single-token calls: after each, every held code is within the steps that its page's scale has grown by."""
    cache, before = _cache(tg, 4, 2, 16, 64, torch.int8)
    table = _table([40], 16, 4, 4)
    g = torch.Generator().manual_seed(9)
    x = (torch.randn(40, 2, 64, generator=g) * torch.linspace(0.1, 3, 40)[:, None, None]).half()
    for i in range(40):
        now = (cache.k.cpu(), cache.k_scale.cpu())
        tg.kv_append(cache, x[i:i + 1].cuda(), x[i:i + 1].cuda(), table.cuda(), _ints([i]))
        units, scales, written = ref.append(x[i:i + 1].double(), *now, table, [i], [1], 16, torch.int8)
        ref.near(cache.k_scale, scales, scales * 2.0 ** -23)
        _check_codes(cache.k, units, written, now[0], torch.int8, 2.0 ** -22, f"step {i}")
    k, _ = tg.kv_read(cache, table.cuda(), _ints([0]), _ints([0, 40]), 40)
    # a value is off by half a step at its writing and by half a step for each time its page's scale grew: the
    # scales grow by the ramp, so the sum of steps is below 16 halves of the last
    err = (k.double().cpu() - x.double()).abs()
    last = torch.stack([cache.k_scale.cpu().double()[int(table[0, t // 16])] for t in range(40)])
    assert (err <= 8.5 * last[:, :, None] + x.double().abs() * 2.0 ** -10).all()


def test_append_in_place_queries_of_a_packed_projection(tg):
    """Queries, keys and values as slices of one projection; the queries rotated where they are."""
    packed = torch.randn(6, (4 + 2 + 2) * 64, generator=torch.Generator().manual_seed(10)).half()
    dev = packed.cuda().view(6, 8, 64)
    cache, before = _cache(tg, 5, 2, 16, 64, torch.float8_e4m3fn)
    table = _table([10, 20], 16, 5, 5)
    f, lens, counts = ref.freqs(64), [8, 16], [2, 4]
    out = tg.kv_append(cache, dev[:, 4:6], dev[:, 6:], table.cuda(), _ints(lens), _ints([0, 2, 6]), max_new=4, Q=dev[:, :4], out=dev[:, :4], inv_freq=f.cuda(),
                       layout=tg.ROPE_INTERLEAVED)
    pos = torch.tensor([8, 9, 16, 17, 18, 19])
    p = packed.view(6, 8, 64)
    want, size = ref.rope(p[:, :4], pos, f, 1.0, True)
    _near_rotated(out, want, size, torch.float16)
    assert torch.equal(dev.cpu()[:, 4:], p[:, 4:])
    units, scales, written = ref.append(p[:, 6:].double(), before[1], before[3], table, lens, counts, 16, torch.float8_e4m3fn)
    _check_codes(cache.v, units, written, before[1], torch.float8_e4m3fn, 2.0 ** -22, "values")
    kd, _ = ref.rope(p[:, 4:6], pos, f, 1.0, True)
    units, scales, written = ref.append(kd, before[0], before[2], table, lens, counts, 16, torch.float8_e4m3fn)
    u = units.clamp(-448, 448)
    assert not (((cache.k.cpu().double() - u).abs() > ref.code_step(u, torch.float8_e4m3fn) / 2 + 448 * 2.0 ** -20) & written).any()


@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("rotary", [0, 2, 32, 48])
def test_append_rotates_part_of_unaligned_keys(tg, rotary, off):
    """Keys and values that begin at any element, the rotated part of a head of any even width."""
    cache, before = _cache(tg, 20, 3, 32, 64, torch.float8_e4m3fn)
    table = _table([200], 32, 20, 6)
    k = torch.randn(150, 3, 64, generator=torch.Generator().manual_seed(12)).bfloat16()
    base = torch.zeros(150 * 200 + 8, dtype=torch.bfloat16, device="cuda")
    x = base[off:off + 150 * 200].view(150, 200)[:, :192].view(150, 3, 64) if not off else base[off:].as_strided((150, 3, 64), (200, 64, 1))
    x.copy_(k)
    f = ref.freqs(rotary) if rotary else None
    tg.kv_append(cache, x, x, table.cuda(), _ints([50]), _ints([0, 150]), max_new=150, inv_freq=f.cuda() if rotary else None)
    kd = ref.rope(k, torch.arange(50, 200), f, 1.0, False)[0] if rotary else k.double()
    units, scales, written = ref.append(kd, before[0], before[2], table, [50], [150], 32, torch.float8_e4m3fn)
    u = units.clamp(-448, 448)
    assert not (((cache.k.cpu().double() - u).abs() > ref.code_step(u, torch.float8_e4m3fn) / 2 + 448 * 2.0 ** -20) & written).any()


READ = [  # firsts, counts, page, heads, dim, cache type, element type
    ([0], [1], 16, 1, 64, 0, 0), ([0, 3, 70], [5, 0, 100], 64, 8, 128, 0, 1), ([1, 17, 33], [33, 64, 7], 16, 3, 64, 1, 0), ([127], [500], 128, 2, 128, 1, 1),
    ([0, 0, 0], [777, 31, 256], 32, 4, 64, 1, 1), ([5, 0, 0, 9], [0, 0, 200, 0], 64, 1, 64, 0, 0),
]


@pytest.mark.parametrize("firsts,counts,page,heads,dim,ct,dt", READ)
def test_read(tg, firsts, counts, page, heads, dim, ct, dt):
    dtype, half = CODES[ct], HALF[dt]
    total = [a + b for a, b in zip(firsts, counts)]
    pages = sum(-(-t // page) for t in total) + 2
    cache, (k, v, ks, vs) = _cache(tg, pages, heads, page, dim, dtype, seed=7)
    table = _table(total, page, pages, 8)
    cu = [0] + torch.tensor(counts).cumsum(0).tolist()
    K, V = tg.kv_read(cache, table.cuda(), _ints(firsts), _ints(cu), sum(counts), dtype=half)
    for got, c, s in ((K, k, ks), (V, v, vs)):
        want = torch.cat([ref.gather(c, s, table[i][:-(-total[i] // page)].long(), total[i])[firsts[i]:] for i in range(len(counts))])
        ref.near(got, want, want.abs() * (ref.half_step(half) + 2.0 ** -23) + 2.0 ** -25)
    _status_ok(tg)


def test_ranges_are_reported_and_not_followed(tg):
    """Page numbers, lengths and offsets out of range, each checked against the bounds by the kernels: nothing is
    written for them, other sequences are served, and the status says so once."""
    cache, before = _cache(tg, 6, 2, 16, 64, torch.int8)
    x = torch.ones(4, 2, 64, dtype=torch.float16).cuda()
    for table, lens, cu in (([[0, 1], [6, 2]], [0, 0], [0, 2, 4]), ([[0, 1], [-1, 2]], [0, 0], [0, 2, 4]), ([[0, 1], [2, 3]], [0, 31], [0, 2, 4]),
                            ([[0, 1], [2, 3]], [0, -1], [0, 2, 4]), ([[0, 1], [2, 3]], [0, 0], [0, 2, 5]), ([[0, 1], [2, 3]], [0, 0], [0, 2, 1])):
        cache.v.copy_(before[1])
        tg.kv_append(cache, x, x, _ints(table), _ints(lens), _ints(cu), max_new=2)
        st, _ = tg.tg_device_status(None)
        assert st == tg.ERR_BOUNDS, (table, lens, cu)
        got = cache.v.cpu()
        assert (got[0, :, :2] == 127).all()
        assert torch.equal(got[1:], before[1][1:]) and torch.equal(got[0, :, 2:], before[1][0, :, 2:])
    K = torch.full((4, 2, 64), 7.0, dtype=torch.float16).cuda()
    for table, lens in (([[0, 1], [6, 2]], [0, 0]), ([[0, 1], [2, 3]], [0, 31]), ([[0, 1], [2, 3]], [0, -2])):
        K.fill_(7.0)
        V = K.clone()
        tg.kv_read(cache, _ints(table), _ints(lens), _ints([0, 2, 4]), 4, out=(K, V))
        st, _ = tg.tg_device_status(None)
        assert st == tg.ERR_BOUNDS
        assert (K[:2] != 7).any() and (K[2 if lens[1] == -2 else 3] == 7).all()
    _status_ok(tg)


def test_append_and_read_past_four_gigabytes(tg):
    """Pages whose codes begin past 2^32 bytes."""
    page, heads, dim = 128, 8, 128
    pages = (1 << 32) // (page * heads * dim) + 64
    k = torch.empty(pages, heads, page, dim, dtype=torch.int8, device="cuda")
    v = torch.empty_like(k)
    ks, vs = torch.ones(pages, heads, device="cuda"), torch.ones(pages, heads, device="cuda")
    cache = tg.KvCache(k, v, ks, vs)
    x = torch.randn(130, heads, dim, generator=torch.Generator().manual_seed(13)).half()
    table = _ints([[pages - 1, pages - 40]])
    tg.kv_append(cache, x.cuda(), x.cuda(), table, _ints([0]), _ints([0, 130]), max_new=130)
    K, V = tg.kv_read(cache, table, _ints([0]), _ints([0, 130]), 130)
    step = torch.cat([x[:128].double().abs().amax((0, 2)).expand(128, -1), x[128:].double().abs().amax((0, 2)).expand(2, -1)]) / 127
    for got in (K, V):
        ref.near(got, x.double(), step[:, :, None] * 0.5001 + x.double().abs() * 2.0 ** -10)
    _status_ok(tg)


def test_other_stream_and_graph(tg):
    """Append, read and rope on a side stream, and captured once and replayed with new contents."""
    cache, before = _cache(tg, 8, 2, 16, 64, torch.float8_e4m3fn)
    table, lens, cu = _table([20, 30], 16, 8, 9).cuda(), _ints([18, 25]), _ints([0, 2, 7])
    x = torch.randn(7, 2, 64, generator=torch.Generator().manual_seed(14)).half()
    f = ref.freqs(64).cuda()
    static = torch.zeros_like(x).cuda()
    places = _ints(list(range(7)))

    def step():
        tg.kv_append(cache, static, static, table, lens, cu, max_new=5)
        r = tg.rope(static, places, f)
        return (r, *tg.kv_read(cache, table, lens, cu, 7))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r, k, v = step()
    static.copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    want, size = ref.rope(x, torch.arange(7), ref.freqs(64), 1.0, False)
    _near_rotated(r, want, size, torch.float16)
    # the zeros written first left the scales of the partly filled pages alone
    units, scales, written = ref.append(x.double(), before[0], before[2], table.cpu(), [18, 25], [2, 5], 16, torch.float8_e4m3fn)
    ref.near(cache.k_scale, scales, scales * 2.0 ** -23)
    _check_codes(cache.k, units, written, before[0], torch.float8_e4m3fn, 2.0 ** -22, "graph")
    side2 = torch.cuda.Stream()
    side2.wait_stream(torch.cuda.current_stream())
    y = tg.rope(static, places, f, stream=side2)
    side2.synchronize()
    assert torch.equal(y, r)


@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("graph", [False, True])
def test_rotated_prompts_are_whole_before_what_follows(tg, graph, off):
    """A rotated append of prompts is several launches side by side: whatever comes behind it on the stream, reading
    or overwriting, meets all of them ended. Every round's results are those of a round with a wait after each call."""
    counts, lens, page, heads, dim = [900, 37, 0, 1400], [10, 64, 5, 0], 64, 4, 128
    T, f = sum(counts), ref.freqs(128).cuda()
    total = [a + b for a, b in zip(counts, lens)]
    pages = sum(-(-t // page) for t in total) + 2
    cache, _ = _cache(tg, pages, heads, page, dim, torch.int8)
    start = [x.clone() for x in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    table, first, cu = _table(total, page, pages, 3).cuda(), _ints(lens), _ints([0, 900, 937, 937, 2337])
    none, every = _ints([0] * 4), _ints([0] + torch.tensor(total).cumsum(0).tolist())
    rounds = 12
    x = torch.randn(rounds, T, 4 * heads + 1, dim, generator=torch.Generator().manual_seed(4)).half().cuda()

    def round_of(i, wait):
        for a, b in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), start):
            a.copy_(b)
        rows = x[i].clone()
        flat = rows.view(T, -1)
        q = torch.as_strided(rows, (T, 2 * heads, dim), (flat.shape[1], dim, 1), 2 * heads * dim + off)
        k, v = rows[:, :heads], rows[:, heads:2 * heads]
        wait()
        out = tg.kv_append(cache, k, v, table, first, cu, max_new=max(counts), Q=q, inv_freq=f)
        wait()
        rows.zero_()  # overwrites what the call reads
        got = (out.clone(), *tg.kv_read(cache, table, none, every, sum(total)))
        wait()
        return got

    want = [round_of(i, torch.cuda.synchronize) for i in range(rounds)]
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = [round_of(i, lambda: None) for i in range(rounds)]
        g.replay()
    else:
        got = [round_of(i, lambda: None) for i in range(rounds)]
    torch.cuda.synchronize()
    for i in range(rounds):
        for a, b in zip(got[i], want[i]):
            assert torch.equal(a, b), i
    _status_ok(tg)
