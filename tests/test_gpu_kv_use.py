"""GPU checks of how the cache operators' tensor forms treat what a program does around them."""
import copy

import pytest
import torch

from tests import test_gpu_attention_kv as attend

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


def _filled(tg, pages=4, kv=2, page=16, dim=64, dtype=torch.int8):
    k, v = ((torch.randint(-100, 101, (pages, kv, page, dim)).float()).to(dtype).cuda() for _ in range(2))
    return tg.KvCache(k, v, *(torch.rand(pages, kv).add(0.5).cuda() / 64 for _ in range(2)))


def test_a_cache_keeps_its_tensors(tg):
    cache = _filled(tg)
    other = _filled(tg)
    for name in ("k", "v", "k_scale", "v_scale", "pages", "kv_heads", "page", "dim", "fmt", "args"):
        with pytest.raises(AttributeError):
            setattr(cache, name, getattr(other, name))
        with pytest.raises(AttributeError):
            delattr(cache, name)
    assert (cache.pages, cache.kv_heads, cache.page, cache.dim, cache.fmt) == (4, 2, 16, 64, tg.KV_INT8)
    assert tg.KvCache.empty(1, 1).fmt == tg.KV_E4M3


def test_a_cache_can_be_copied(tg):
    cache = _filled(tg)
    same, other = copy.copy(cache), copy.deepcopy(cache)
    assert all(a is b for a, b in zip(same.args, cache.args))
    other.k.zero_()
    assert (cache.k != 0).any() and torch.equal(other.v, cache.v) and other.v.data_ptr() != cache.v.data_ptr()
    assert (tg.kv_read(other, _ints([[0]]), _ints([0]), _ints([0, 9]), 9)[0] == 0).all()


def test_a_cache_whose_storage_was_exchanged(tg):
    """The kernels see what the tensors hold at the call; a shape that no longer fits is refused."""
    cache, other = _filled(tg), _filled(tg, pages=9)
    table, q = _ints([[1, 3]]), torch.randn(1, 2, 64).half().cuda()
    args = (table, _ints([0]), _ints([0, 20]), 20)
    for a, b in zip(cache.args, other.args):
        a.data = b.data
    assert cache.pages == 9
    for a, b in zip(tg.kv_read(cache, *args), tg.kv_read(other, *args)):
        assert torch.equal(a, b)
    assert torch.equal(tg.attention_kv(q, cache, table, _ints([20])), tg.attention_kv(q, other, table, _ints([20])))
    cache.v_scale.data = torch.zeros(8, 2, device="cuda")
    with pytest.raises(ValueError, match="scales must have shape"):
        tg.kv_read(cache, *args)
    _status_ok(tg)


# ---------------------------------------------------------------- rows that no sequence has

NOTHING = [[0, 3, 5], [2, 5, 7], [3, 3, 3], [9, 9, 9], [0, 0, 0], [0]]   # of nine rows: padded behind, around, empty, no sequences


@pytest.mark.parametrize("wide", [1, 40])  # the kernels for few rows, and for many
@pytest.mark.parametrize("offsets", NOTHING)
@pytest.mark.parametrize("dim", [64, 128])
def test_attention_of_rows_that_no_sequence_has(tg, wide, offsets, dim):
    cache = _filled(tg, pages=40, dim=dim)
    batch, offsets = len(offsets) - 1, [wide * x for x in offsets]
    T = 9 * wide
    lens = _ints([5 * wide, 100 + wide][:batch])
    table = torch.arange(40, dtype=torch.int32).view(2, 20)[:batch].cuda()
    q = torch.randn(T, 4, dim, generator=torch.Generator().manual_seed(1)).half().cuda()
    out = torch.full_like(q, torch.nan)
    got, lse = tg.attention_kv(q, cache, table, lens, _ints(offsets), max_new=5 * wide, max_len=320, out=out, return_lse=True)
    fresh = tg.attention_kv(q, cache, table, lens, _ints(offsets), max_new=5 * wide, max_len=320)
    _status_ok(tg)
    none = torch.ones(T, dtype=torch.bool, device="cuda")
    none[offsets[0]:offsets[-1]] = False
    assert (got[none] == 0).all() and (lse[none] == -torch.inf).all() and torch.equal(got, fresh)
    assert got.isfinite().all() and lse[~none].isfinite().all() and (got[~none] != 0).any(-1).all()


@pytest.mark.parametrize("most", [2, 70])
@pytest.mark.parametrize("max_len", [64, 4000])
def test_attention_of_spans_out_of_range(tg, most, max_len):
    """Reported, and zeros in their rows whatever the output held; the other sequences are as they were."""
    cache = _filled(tg, pages=16)
    table, lens = torch.arange(16, dtype=torch.int32).view(4, 4).cuda(), _ints([60, 64, 50, 64])
    cu = [i * most for i in range(5)]
    q = torch.randn(4 * most, 8, 64, generator=torch.Generator().manual_seed(2)).half().cuda()

    def run(offsets, bound):
        out = torch.full_like(q, torch.nan)
        return tg.attention_kv(q, cache, table, lens, _ints(offsets), max_new=bound, max_len=max_len, out=out, return_lse=True)

    good, glse = run(cu, most)
    _status_ok(tg)
    for offsets, bound, zero, same in ((cu[:2] + [cu[2] + 1] + cu[3:], most, (most, 2 * most + 1), (0, most)),          # longer than max_new
                                       (cu[:4] + [cu[4] + 1], most + 1, (3 * most, 4 * most), (0, 3 * most)),           # past the end
                                       ([-1] + cu[1:], most + 2, (0, most), (most, 4 * most))):                         # before the start
        out, lse = run(offsets, bound)
        assert tg.tg_device_status(None)[0] == tg.ERR_BOUNDS, offsets
        assert (out[slice(*zero)] == 0).all() and (lse[slice(*zero)] == -torch.inf).all(), offsets
        near = dict(rtol=2.0 ** -9, atol=2.0 ** -12)   # the work may be split in another way
        assert torch.allclose(out[slice(*same)], good[slice(*same)], **near) and torch.allclose(lse[slice(*same)], glse[slice(*same)], **near)
        assert out.isfinite().all()
    _status_ok(tg)


@pytest.mark.parametrize("offsets", NOTHING)
def test_reading_rows_that_no_sequence_has(tg, offsets):
    cache = _filled(tg)
    batch = len(offsets) - 1
    table, first = _ints([[0, 1], [2, 3]])[:batch], _ints([1, 15])[:batch]
    out = tuple(torch.full((9, 2, 64), torch.nan, dtype=torch.float16, device="cuda") for _ in range(2))
    tg.kv_read(cache, table.contiguous(), first, _ints(offsets), 9, out=out)
    _status_ok(tg)
    none = torch.ones(9, dtype=torch.bool, device="cuda")
    none[offsets[0]:offsets[-1]] = False
    for x in out:
        assert (x[none] == 0).all() and x.isfinite().all() and (x[~none] != 0).any(-1).all()


@pytest.mark.parametrize("most", [1, 3])      # the kernels for single tokens, and for prompts
@pytest.mark.parametrize("off", [0, 1])       # whole 16-byte pieces, and not
@pytest.mark.parametrize("case", [([0, 1, 2], [0, 0], 0), ([2, 3, 4], [5, 31], 0), ([5, 5, 5], [0, 0], 0), ([0], [], 0),
                                  ([1, 2, 3], [32, 3], 1), ([1, 2, 3], [-1, 3], 1), ([1, 9, 8], [0, 3], 1), ([1, 6, 7], [3, 3], 1)])
def test_queries_that_are_not_rotated_are_copied(tg, most, off, case):
    """Rows of no sequence, and of a sequence that is out of range (reported)."""
    offsets, lens, bad = case
    if most > 1:
        offsets, lens = [most * x for x in offsets], [x if x != 31 else 29 for x in lens]
    T, batch = 7 * most, len(lens)
    cache = _filled(tg, pages=4)
    table = _ints([[0, 1], [2, 3]])[:batch].contiguous()
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn(T, 2, 64, generator=g).half().cuda() for _ in range(2))
    q = torch.randn(T * 4 * 64 + 8, generator=g).half().cuda()[off:off + T * 256].view(T, 4, 64)
    f, amplitude = tg.rope_frequencies(64)
    out = torch.full((T, 4, 64), torch.nan, dtype=torch.float16, device="cuda")
    tg.kv_append(cache, k, v, table, _ints(lens), _ints(offsets), max_new=most, Q=q, inv_freq=f, amplitude=2.0, out=out)
    assert tg.tg_device_status(None)[0] == (tg.ERR_BOUNDS if bad else tg.OK)
    want, row = q.clone(), 0
    for i in range(batch):
        lo, hi = offsets[i], offsets[i + 1]
        if 0 <= lo < hi <= T and hi - lo <= most and lens[i] >= 0 and lens[i] + hi - lo <= 32:
            want[lo:hi] = tg.rope(q[lo:hi], torch.arange(lens[i], lens[i] + hi - lo, dtype=torch.int32, device="cuda"), f, 2.0)
    turned = (want != q).any(-1).any(-1)
    assert torch.equal(out[~turned], q[~turned])
    assert torch.allclose(out[turned].float(), want[turned].float(), rtol=2.0 ** -10, atol=2.0 ** -16)
    inplace = q.clone()
    tg.kv_append(cache, k, v, table, _ints(lens), _ints(offsets), max_new=most, Q=inplace, inv_freq=f, amplitude=2.0, out=inplace)
    tg.tg_device_status(None)
    assert torch.equal(inplace[~turned], q[~turned])
    _status_ok(tg)


# ---------------------------------------------------------------- one page of several out of range

@pytest.mark.parametrize("entry", [4, -1, 2 ** 31 - 1])
@pytest.mark.parametrize("rotate", [False, True])
def test_append_with_the_second_of_three_pages_out_of_range(tg, entry, rotate):
    """That page's tokens are not written; the sequence's others are, as without the fault, and its queries are rotated."""
    g = torch.Generator().manual_seed(4)
    k, v = (torch.randn(45, 2, 64, generator=g).half().cuda() for _ in range(2))
    q = torch.randn(45, 4, 64, generator=g).half().cuda()
    f, _ = tg.rope_frequencies(64)
    start = _filled(tg)
    caches, outs = [], []
    for second in (2, entry):
        cache = tg.KvCache(*(x.clone() for x in start.args))
        outs.append(tg.kv_append(cache, k, v, _ints([[3, second, 1]]), _ints([2]), _ints([0, 45]), max_new=45, Q=q if rotate else None,
                                 inv_freq=f if rotate else None))
        assert tg.tg_device_status(None)[0] == (tg.OK if second == 2 else tg.ERR_BOUNDS)
        caches.append(cache)
    for whole, part, before in zip(caches[0].args, caches[1].args, start.args):
        assert torch.equal(part[[1, 3]], whole[[1, 3]]) and torch.equal(part[[0, 2]], before[[0, 2]])
        assert not torch.equal(whole[2], before[2])
    if rotate:
        assert torch.equal(*outs)
    _status_ok(tg)


# ---------------------------------------------------------------- what torch is told

def test_tensors_that_are_overwritten_say_so(tg):
    cache = _filled(tg)
    k, q = torch.randn(1, 2, 64).half().cuda(), torch.randn(1, 4, 64).half().cuda()
    f, _ = tg.rope_frequencies(64)
    table, lens = _ints([[0, 1]]), _ints([3])

    def bumped(call, changed, kept):
        before = [x._version for x in (*changed, *kept)]
        call()
        after = [x._version for x in (*changed, *kept)]
        assert [a > b for a, b in zip(after, before)] == [True] * len(changed) + [False] * len(kept)

    pair = (torch.empty_like(k), torch.empty_like(k))
    o = torch.empty_like(q)
    bumped(lambda: tg.kv_append(cache, k, k, table, lens, Q=q, inv_freq=f, out=q), (*cache.args, q), (k, table, lens, f))
    bumped(lambda: tg.kv_append(cache, k, k, table, lens, Q=q, inv_freq=f), cache.args, (k, q))
    bumped(lambda: tg.rope(q, lens, f, out=q), (q,), (lens, f))
    bumped(lambda: tg.rope(q, lens, f), (), (q, lens, f))
    bumped(lambda: tg.kv_read(cache, table, lens, None, 1, out=pair), pair, cache.args)
    bumped(lambda: tg.attention_kv(q, cache, table, lens, out=o), (o,), (q, *cache.args))
    x = torch.randn(1, 4, 64, device="cuda", requires_grad=True)
    y = x.half().exp()   # the gradient of exp reads its output
    tg.rope(y.detach(), lens, f, out=y.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    with torch.inference_mode():
        frozen = _filled(tg)
    tg.kv_append(frozen, k, k, table, lens)  # tensors that torch keeps no account of
    _status_ok(tg)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("backward", [False, True])
def test_rope_has_a_gradient(tg, interleaved, backward):
    """The gradient of a weighted sum is the transposed rotation of the weights, and so are those of slices, of a plain
    sum (whose gradient is one value, spread) and on another stream."""
    g = torch.Generator().manual_seed(6)
    packed = torch.randn(5, 6, 64, generator=g).half().cuda().requires_grad_()
    w = torch.randn(5, 4, 64, generator=g).half().cuda()
    pos = _ints([3, 1, 4, 1, 5])
    f, _ = tg.rope_frequencies(32)
    how = dict(amplitude=1.25, layout=tg.ROPE_INTERLEAVED if interleaved else tg.ROPE_HALF)

    def gradient(weight, stream=None):
        y = tg.rope(packed[:, 1:5], pos, f, backward=backward, stream=stream, **how)
        assert y.requires_grad and torch.equal(y, tg.rope(packed.detach()[:, 1:5], pos, f, backward=backward, **how))
        if stream is not None:
            torch.cuda.current_stream().wait_stream(stream)
        (d,) = torch.autograd.grad((y * weight).sum() if weight is not None else y.sum(), packed)
        assert (d[:, [0, 5]] == 0).all()
        return d[:, 1:5]

    want = tg.rope(w, pos, f, backward=not backward, **how)
    assert torch.equal(gradient(w), want)
    assert torch.equal(gradient(None), tg.rope(torch.ones_like(w), pos, f, backward=not backward, **how))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert torch.equal(gradient(w, side), want)
    x = packed[:, 1:5]
    with pytest.raises(RuntimeError, match="no gradient"):
        tg.rope(x, pos, f, out=torch.empty_like(x))
    with torch.no_grad():
        assert not tg.rope(x, pos, f).requires_grad
    # the gradient's own gradient: the map is linear, so that of <w, rope(x)> by w is rope(x)
    w.requires_grad_()
    y = tg.rope(packed[:, 1:5], pos, f, backward=backward, **how)
    (d,) = torch.autograd.grad(y, packed, w, create_graph=True)
    (dw,) = torch.autograd.grad(d, w, packed.detach())
    assert torch.equal(dw, y)
    _status_ok(tg)


def test_layouts_are_not_cut_to_32_bits(tg):
    x, pos = torch.zeros(1, 1, 64).half().cuda(), _ints([0])
    f, _ = tg.rope_frequencies(64)
    for layout in (1 << 32, -(1 << 32) + 1):
        with pytest.raises(ValueError, match="layout"):
            tg.rope(x, pos, f, layout=layout)
        with pytest.raises(ValueError, match="layout"):
            tg.kv_append(_filled(tg, kv=1), x, x, _ints([[0]]), pos, inv_freq=f, layout=layout)
    for layout in (2, -1):
        with pytest.raises(tg.TgError, match="layout"):
            tg.rope(x, pos, f, layout=layout)


# ---------------------------------------------------------------- scales that no append writes

@pytest.mark.parametrize("most", [1, 4, 70])
@pytest.mark.parametrize("which", [2, 3])
def test_a_scale_that_is_nan_reaches_the_rows_that_see_it(tg, most, which):
    cache, host, table, q = attend._case(tg, [most, most], [most + 90, most + 90], 16, 2, 4, 64, 0, 0, seed=42, garbage=False)
    cache.args[which][int(table[0, 3]), 1] = torch.nan
    out = tg.attention_kv(q.cuda(), cache, table.cuda(), _ints([most + 90] * 2), _ints([0, most, 2 * most]), max_new=most, max_len=most + 90)
    assert out[:most, 4:].isnan().all() and not out[:most, :4].isnan().any() and not out[most:].isnan().any()
    _status_ok(tg)
