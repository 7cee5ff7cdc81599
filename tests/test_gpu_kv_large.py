"""GPU checks of the cache operators at sizes where a CTA makes many rounds: against the definitions in float64 of the
small tests, the same bits from launch to launch, and waits that run out."""
import pytest
import torch

from tests import kv_reference as ref
from tests import test_gpu_attention_kv as attend
from tests import test_gpu_kv_cache as cache_tests

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


def _status_ok(tg):
    st, where = tg.tg_device_status(None)
    assert st == tg.OK, f"device status {st} at {where}"


def _made_on_the_gpu(tg, counts, lens, page, kv, share, dim, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    need = [-(-n // page) for n in lens]
    order = torch.randperm(sum(need), generator=g, device="cuda").int()
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, m in enumerate(need):
        table[i, :m] = order[at:at + m]
        at += m
    k, v = (torch.randint(-100, 101, (at, kv, page, dim), generator=g, dtype=torch.int8, device="cuda") for _ in range(2))
    if dtype is not torch.int8:
        k, v = ((x.half() * 4).to(dtype) for x in (k, v))
    ks, vs = (torch.rand(at, kv, generator=g, device="cuda").add(0.5) / (70 if dtype is torch.int8 else 280) for _ in range(2))
    q = torch.randn(sum(counts), kv * share, dim, generator=g, device="cuda").half()
    return tg.KvCache(k, v, ks, vs), table, q


@pytest.mark.parametrize("batch,most,longest,page,share,dim,dtype", [
    (64, 1, 8000, 64, 4, 128, torch.float8_e4m3fn),   # a decode step: every ring slot filled some twenty times
    (33, 5, 6000, 16, 7, 64, torch.int8),             # drafts
    (2, 2048, 6000, 64, 4, 128, torch.float8_e4m3fn),  # prompt chunks
    (3, 600, 3000, 16, 3, 64, torch.int8),
])
def test_forty_launches_agree_bit_for_bit(tg, batch, most, longest, page, share, dim, dtype):
    """A slot of codes is refilled by the copy engine after ordinary reads; a copy that overtook them would show as
    other results from launch to launch."""
    r = torch.Generator().manual_seed(batch)
    lens = [longest - int(torch.randint(0, longest // 2, (), generator=r)) for _ in range(batch)]
    counts = [most - int(torch.randint(0, most // 2 + 1, (), generator=r)) for _ in range(batch)]
    counts[0] = most
    cache, table, q = _made_on_the_gpu(tg, counts, lens, page, 8, share, dim, dtype, seed=batch)
    cu = _ints([0] + torch.tensor(counts).cumsum(0).tolist())

    def once():
        return tg.attention_kv(q, cache, table, _ints(lens), cu, max_new=most, max_len=longest, return_lse=True)

    out, lse = once()
    assert out.isfinite().all() and lse.isfinite().all()
    for i in range(39):
        again, lagain = once()
        assert torch.equal(out, again) and torch.equal(lse, lagain), f"launch {i + 2} differs"
    _status_ok(tg)


# ---------------------------------------------------------------- many rounds of a CTA

@pytest.mark.parametrize("counts,lens,page,heads,dim,ct,dt", [
    ([9000, 1, 6000, 5003], [5, 63, 0, 130], 64, 8, 64, 0, 0),   # a CTA takes four heads of a page one after another
    ([7001, 5000], [17, 16], 16, 8, 64, 1, 1),                   # eight, four at a time
    ([300, 8200], [77, 0], 32, 16, 128, 1, 0),
])
@pytest.mark.parametrize("rotate", [False, True])
def test_append_of_many_heads_a_cta(tg, counts, lens, page, heads, dim, ct, dt, rotate):
    cache_tests.test_append(tg, counts, lens, page, heads, dim, ct, dt, True, rotate)


@pytest.mark.parametrize("counts,lens,page,kv,share,dim,ct,dt", [
    ([1, 1, 1], [200000, 170001, 199999], 128, 4, 4, 64, 1, 0),  # over 64 steps a warp and unit: pages and scales are fetched three times
    ([3, 2, 3], [200000, 199990, 190007], 16, 2, 4, 64, 0, 1),   # over 32, blocks of 16 rows
    ([1] * 12, [60000] * 11 + [59000], 64, 2, 2, 128, 0, 0),
])
def test_attention_over_many_steps(tg, counts, lens, page, kv, share, dim, ct, dt):
    cache, host, table, q = attend._case(tg, counts, lens, page, kv, share, dim, ct, dt, seed=31)
    cu = [0] + torch.tensor(counts).cumsum(0).tolist()
    out, lse = tg.attention_kv(q.cuda(), cache, table.cuda(), _ints(lens), _ints(cu), max_new=max(counts), max_len=max(lens), return_lse=True)
    attend._check(out, lse, host, table, q, counts, lens, page, True, 0, dim ** -0.5)
    _status_ok(tg)


def test_prompt_chunks_of_more_sequences_than_threads(tg):
    """Most of 900 sequences have one new token, some 70, a few are idle: the chunk kernel's list takes two passes."""
    g = torch.Generator().manual_seed(32)
    lens = [int(n) for n in torch.randint(1, 200, (900,), generator=g)]
    counts = [1] * 900
    for i in (0, 500, 767, 768, 899):
        counts[i], lens[i] = 70, 100 + i % 60
    for i in (3, 770, 771):
        lens[i] = 0
    counts[770] = 0
    cache, host, table, q = attend._case(tg, counts, lens, 16, 2, 1, 64, 0, 0, seed=33)
    cu = [0] + torch.tensor(counts).cumsum(0).tolist()
    out, lse = tg.attention_kv(q.cuda(), cache, table.cuda(), _ints(lens), _ints(cu), max_new=70, max_len=200, return_lse=True)
    attend._check(out, lse, host, table, q, counts, lens, 16, True, 0, 0.125)
    _status_ok(tg)


# ---------------------------------------------------------------- many small weights under a few large ones

@pytest.mark.parametrize("batch,most,ct", [(2000, 1, 1), (700, 3, 0), (200, 70, 1), (60, 260, 0)])
def test_small_weights_under_large_ones_count(tg, batch, most, ct):
    """Four keys of zero value (one for each warp of the kernel for few rows) take all but about 2^-14.6 of a row's
    weight, so each of the 8188 others, whose values are all positive and make up the whole output, has some 2^-25.6
    of the largest weight. All sequences have the same pages, so that a CTA walks a sequence whole.

    A weight is rounded to 16 bits: by 2^-11 of itself, or by 2^-34 of the row's largest."""
    L, dim, page, dtype = 8192, 64, 64, attend.CODES[ct]
    g = torch.Generator().manual_seed(most)
    sign = torch.randint(0, 2, (dim,), generator=g) * 2 - 1
    k = torch.randint(-10, 11, (L, dim), generator=g)
    v = torch.randint(50, 121, (L, dim), generator=g) // 8 * 8   # exact in e4m3
    sinks = [5, 21, 37, 53]
    k[sinks], v[sinks] = 120 * sign, 0
    order = torch.randperm(L // page, generator=g)
    codes = [torch.empty(L // page, 1, page, dim).index_copy_(0, order, x.float().view(L // page, 1, page, dim)).to(dtype) for x in (k, v)]
    # a sink's score: 120 * 64 / 8 * scale = 17.76 = ln(2^25.6) above the others', which are about 0
    scales = [torch.full((L // page, 1), 17.76 / 960), torch.ones(L // page, 1)]
    rows = batch * most
    q = (sign * (1 + torch.rand(rows, 1, 1, generator=g) / 64)).half()
    cache = tg.KvCache(*(x.cuda() for x in codes + scales))
    table = order.int().expand(batch, -1).contiguous().cuda()
    cu = torch.arange(0, rows + 1, most, dtype=torch.int32).cuda()
    out, lse = tg.attention_kv(q.cuda(), cache, table, _ints([L] * batch), cu, max_new=most, max_len=L, return_lse=True)
    _status_ok(tg)
    kd, vd = (x.double()[order].view(L, dim).cuda() for x in codes)
    z = q[:, 0].double().cuda() @ (kd * scales[0][0, 0].double()).T / 8
    z = z.masked_fill((torch.arange(L) > L - most + torch.arange(rows)[:, None] % most).cuda(), -torch.inf)
    size = 1.05 * 17.76   # of the largest sum of |q k|, scaled
    ds = 2 * dim * 2.0 ** -24 * size + 2.0 ** -21
    l = torch.logsumexp(z, 1)
    p = (z - l[:, None]).exp()
    o = p @ vd
    small = 2.0 ** -34 * p.amax(1, keepdim=True) * vd.sum(0)
    tol = (2 * ds + 2.0 ** -11 + L * 2.0 ** -24) * o + small
    assert (tol < o * 2.0 ** -7).all()
    ref.near(out[:, 0], o.cpu(), (tol + o * 2.0 ** -11 + 2.0 ** -25).cpu())
    ref.near(lse[:, 0], l.cpu(), (ds + L * 2.0 ** -24 + 2.0 ** -21 * (1 + l.abs())).cpu())


@pytest.mark.parametrize("most", [1, 5, 70])
@pytest.mark.parametrize("dim", [64, 128])
def test_log_of_the_sum_of_equal_weights(tg, most, dim):
    """With a scale of 0 the log of a row's sum is that of the number of its keys, whatever the value scales that the weights
    carry: within the reference's tolerance, of roundings of numbers below 16 and one unit of 2^-24 a key."""
    lens = [most, most + 1, most + 29, most + 200, most + 3000]
    for ct in (0, 1):
        cache, host, table, q = attend._case(tg, [most] * 5, lens, 16, 2, 3, dim, ct, 1, seed=45, garbage=False)
        cu = [most * i for i in range(6)]
        out, lse = tg.attention_kv(q.cuda(), cache, table.cuda(), _ints(lens), _ints(cu), max_new=most, max_len=max(lens), scale=0.0, return_lse=True)
        attend._check(out, lse, host, table, q, [most] * 5, lens, 16, True, 0, 0.0)
        keys = torch.cat([torch.arange(n - most + 1, n + 1) for n in lens]).double()
        ref.near(lse, keys.log()[:, None].expand(-1, 6), (2.0 ** -20 + keys * 2.0 ** -24 + 2.0 ** -21 * keys.log())[:, None])
    _status_ok(tg)


# ---------------------------------------------------------------- waits that run out

def _times_out_and_recovers(tg, counts, lens, share, dim, max_len):
    """A call with one arrival a CTA withheld ends with a timeout; the next call is what it was before. The
    workspace holds all ones, so that an entry which no kernel wrote would read as sizes far out of range."""
    cache, table, q = _made_on_the_gpu(tg, counts, lens, 16, 2, share, dim, torch.int8, seed=5)
    cu = _ints([0] + torch.tensor(counts).cumsum(0).tolist())
    args = (q, cache, table, _ints(lens), cu)
    want = tg.attention_kv(*args, max_new=max(counts), max_len=max_len)
    _status_ok(tg)
    T, H = q.shape[:2]
    need = tg.tg_attention_kv_workspace(cache.kv_heads, cache.page, dim, cache.fmt, H, len(lens), T, max(counts), max_len, 0, tg.FP16)
    work = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    out, lens_d = torch.empty_like(want), args[3]
    sizes = (cache.pages, cache.kv_heads, cache.page, dim, cache.fmt)
    tg.tg_set_watchdog_ns(20_000_000)  # 20 ms
    tg.tg_debug_skip_first_arrive(True)
    try:
        tg.tg_attention_kv(q.data_ptr(), *q.stride()[:2], out.data_ptr(), None, cache.k.data_ptr(), cache.v.data_ptr(), cache.k_scale.data_ptr(),
                           cache.v_scale.data_ptr(), *sizes, table.data_ptr(), table.shape[1], lens_d.data_ptr(), cu.data_ptr(), len(lens), T, H,
                           max(counts), max_len, 1, 0, dim ** -0.5, tg.FP16, work.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
        st, where = tg.tg_device_status(None)
    finally:
        tg.tg_debug_skip_first_arrive(False)
        tg.tg_set_watchdog_ns(0)
    assert st == tg.ERR_TIMEOUT
    _status_ok(tg)
    assert torch.equal(tg.attention_kv(*args, max_new=max(counts), max_len=max_len), want)
    _status_ok(tg)
    return where


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("counts,lens,share", [
    ([100], [100], 1),                 # one tile a unit
    ([300, 90, 200], [300, 4000, 2111], 4),  # units in parts, several segments a CTA
    ([65] * 40, [700] * 40, 2),        # whole units, one after another
])
def test_withheld_arrivals_of_prompt_chunks_time_out(tg, counts, lens, share, dim):
    where = _times_out_and_recovers(tg, counts, lens, share, dim, max(lens))
    assert where in (1, 2, 3, 4, 6, 7), where  # whichever of the CTAs' waits gave up first


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("counts,lens,share", [
    ([1], [40], 4),                  # one step
    ([1, 5, 3], [300, 9000, 2111], 4),  # units in parts
    ([1] * 300, [200] * 300, 8),     # whole units, one after another
])
def test_withheld_arrivals_of_few_rows_time_out(tg, counts, lens, share, dim):
    assert _times_out_and_recovers(tg, counts, lens, share, dim, max(lens)) == 6  # the wait for a step's codes
