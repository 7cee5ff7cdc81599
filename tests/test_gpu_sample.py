"""GPU checks of drawing tokens, against the definition in 64 bits on the CPU: whole numbers, equal or wrong. The sums of
a row in 64 bits are good to 2^-35 of themselves (2^18 additions of 2^-53 each), the kernel's weights to 2^-37 of
themselves: where a border (of the mass, or of u) lies nearer than 2^-34 of the sum to a token's edge either token may
be right, and a test's inputs have none such. Weights that are whole are exact on both sides."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
NEAR = 2.0 ** -34


@pytest.fixture(scope="module")
def tg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import tiled_tensor_core_tcgen05_gb300 as m
    torch.cuda.set_device(0)
    return m


def draw(x, u, t, k, p, m):
    """(token, whether it is beyond doubt) of one row, float64."""
    x = torch.where(x.isnan(), -math.inf, x.double())
    top = float(x.max())
    if top == -math.inf:
        return -1, True
    if not t > 0:
        return int((x == top).nonzero()[0]), True
    y = torch.where(x == top, 0.0, (x - top) / t if top < math.inf else torch.full_like(x, -math.inf))
    y = torch.where(x == -math.inf, -math.inf, y)
    y, at = y.sort(descending=True, stable=True)
    keep = y > -math.inf
    if k > 0:
        keep[k:] = False
    if m > 0:
        keep &= y >= math.log(min(m, 1.0))
    w = y.exp() * keep
    w = torch.where(w < 2.0 ** -43, 0.0, w)  # less than half a unit of the weights is none
    whole = bool((w == w.round()).all())
    sure = True
    if p < 1:
        before = w.cumsum(0) - w
        edge = max(p, 0.0) * float(w.sum())
        sure &= whole or bool(((before[keep][1:] - edge).abs() > NEAR * w.sum()).all())  # the first is kept in any case
        ok = before < edge
        ok[0] = True
        w = w * ok
    c = torch.zeros_like(w).scatter_(0, at, w).cumsum(0)
    edge = min(max(u, 0.0), 1 - 2.0 ** -24) * float(c[-1])
    sure &= whole or edge == 0 or bool(((c - edge).abs() > NEAR * c[-1]).all())
    return int((c > edge).nonzero()[0]), sure


def _check(tg, x, u, t=None, k=None, p=None, m=None, **how):
    """x, u on the CPU; settings numbers, or lists of one a row."""
    rows = x.shape[0]
    on = lambda v, d: torch.tensor(v, dtype=d, device="cuda") if isinstance(v, list) else v  # noqa: E731
    out = torch.full((rows,), -7, dtype=torch.int32, device="cuda")  # that every row writes
    got = tg.sample(how.get("device_x", x.cuda()), u.cuda(), on(t, torch.float32), on(k, torch.int32), on(p, torch.float32), on(m, torch.float32), out=out)
    assert got.dtype is torch.int32 and tuple(got.shape) == (rows,)

    def of(v, i, none):  # in 32 bits, as the call has it
        v = v[i] if isinstance(v, list) else v
        return none if v is None else v if isinstance(v, int) else float(torch.tensor(v, dtype=torch.float32))

    for i, token in enumerate(got.tolist()):
        want, sure = draw(x[i], float(u[i]), of(t, i, 1.0), of(k, i, 0), of(p, i, 1.0), of(m, i, 0.0))
        assert sure, f"row {i}: a border too near to a token's edge to say"
        assert token == want, f"row {i}: {token}, not {want}"
    return got


def _logits(rows, vocab, dtype, spread=2.5, seed=0):
    g = torch.Generator().manual_seed(seed + vocab)
    x = torch.randn(rows, vocab, generator=g) * spread
    x.scatter_add_(1, torch.randint(0, vocab, (rows, 8), generator=g), torch.rand(rows, 8, generator=g) * 4 * spread)
    return x.to(dtype), torch.rand(rows, generator=g)


TYPES = [torch.float16, torch.bfloat16, torch.float32]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [1, 2, 3, 31, 257, 4099, 32000, 131071])
def test_settings(tg, dtype, vocab):
    """A row of each mixture of settings."""
    some = [(t, k, p, m) for t in (0.0, 0.4, 1.0, 3.0) for k in (0, 1, 7, 900, 5000) for p in (1.0, 0.9, 0.3) for m in (0.0, 0.05)]
    x, u = _logits(len(some), vocab, dtype)
    _check(tg, x, u, *(list(v) for v in zip(*some)))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("spread", [0.0, 0.01, 0.5, 8.0, 60.0])
@pytest.mark.parametrize("rows,vocab", [(1, 40000), (9, 131072), (400, 3001)])
def test_flat_and_steep_rows(tg, dtype, spread, rows, vocab):
    """From all logits alike (ties by index everywhere) to a single token that counts."""
    x, u = _logits(rows, vocab, dtype, spread)
    for k, p, m in ((None, None, None), (None, 0.95, None), (None, 0.05, None), (2999, None, None), (2999, 0.5, None), (None, 0.999, 0.01)):
        _check(tg, x, u, None, k, p, m)


def test_many_ties_at_every_border(tg):
    g = torch.Generator().manual_seed(4)
    x = torch.randint(-3, 4, (12, 50001), generator=g).float()
    x[:, 100:40000] = 2.0
    x[6:, :] = torch.randint(0, 2, (6, 50001), generator=g).float() * 1e-3
    u = torch.rand(12, generator=g)
    for k, p in ((None, 0.5), (12345, None), (45000, 0.77), (1, None), (2000, 0.9), (None, 0.001)):
        _check(tg, x, u, None, k, p, None)


def test_every_token_of_a_small_row_is_drawn_as_often_as_it_should_be(tg):
    """u on a grid: each token's count is its share of the grid, to one."""
    x = torch.tensor([0.3, -1.0, 2.0, -math.inf, 1.1, 2.0, math.nan, -0.0])
    n = 4096
    u = (torch.arange(n) + 0.5) / n
    got = tg.sample(x.repeat(n, 1).cuda(), u.cuda(), temperature=0.7).cpu()
    p = torch.softmax(torch.where(x.isnan(), -math.inf, x.double()) / 0.7, 0)
    count = torch.bincount(got.long(), minlength=8)
    assert ((count - n * p).abs() <= 1).all() and count[3] == count[6] == 0
    assert bool((got[1:] >= got[:-1]).all())


@pytest.mark.parametrize("dtype", TYPES)
def test_infinities_nan_and_empty_rows(tg, dtype):
    inf, nan = math.inf, math.nan
    rows = [[-inf] * 6, [nan] * 6, [nan, -inf, 1.0, -inf, nan, 0.5], [inf, 1.0, inf, -inf, nan, inf], [0.0, -0.0, 0.0, -0.0, -1.0, -inf], [-5e4, 5e4, -5e4, 5e4, 0.0, 1.0],
            [-inf, -inf, -6e4, -inf, -inf, -inf], [inf, inf, inf, inf, inf, inf]]
    x = torch.tensor(rows).to(dtype)
    for u in (0.0, 0.3, 0.55, 0.99999994):
        for t in (None, 0.0, 1e-3, 50.0, 1e30):
            _check(tg, x, torch.full((len(rows),), u), t, None, None, None)
            _check(tg, x, torch.full((len(rows),), u), t, 2, 0.9, None)
            _check(tg, x, torch.full((len(rows),), u), t, None, None, 0.5)


def test_u_and_settings_beyond_their_range(tg):
    x, _ = _logits(6, 500, torch.float32)
    u = torch.tensor([-1.0, 1.0, 7.0, math.inf, 0.0, 0.5])
    _check(tg, x, u)
    _check(tg, x, u, k=[500, 501, 2 ** 31 - 1, -4, 0, 499])
    _check(tg, x, u, p=[0.0, -1.0, 1.0, 2.0, 1e-20, 1e-30])
    _check(tg, x, u, m=[1.0, 2.0, 1e-30, -1.0, 0.9999, 1e30])
    _check(tg, x, u, t=[-1.0, 1e-38, 1e38, math.inf, 1e-45, 1.0])
    nan = torch.full((6,), math.nan, device="cuda")
    got = tg.sample(x.cuda(), nan)
    assert torch.equal(got, tg.sample(x.cuda(), torch.zeros(6, device="cuda")))
    assert torch.equal(tg.sample(x.cuda(), u.cuda(), temperature=nan).cpu().long(), x.argmax(1))
    assert torch.equal(tg.sample(x.cuda(), u.cuda(), top_p=nan, min_p=nan), tg.sample(x.cuda(), u.cuda()))


def test_large_logits_far_apart(tg):
    x, u = _logits(4, 9000, torch.float32, 1e37)
    x[2] = 3e38
    x[3, ::2] = -3e38
    _check(tg, x, u, 5e36)
    _check(tg, x, u, 5e36, 40, 0.9)


@pytest.mark.parametrize("p", [None, 0.9])
@pytest.mark.parametrize("t", [1e-45, 1e-38, 1e-8, 0.002, 0.03, 0.06, 0.1, 0.5])
def test_logits_as_coarse_as_the_temperature(tg, t, p):
    """Neighbours of the largest logit (steps of 2^-7 in bfloat16 there, 2^-10 in float16, 2^-23 and 2^4 in float32) from all alike to none beside it."""
    g = torch.Generator().manual_seed(13)
    for top, dtype in ((1.0, torch.bfloat16), (-1.9, torch.float16), (1.5, torch.float32), (1e8, torch.float32), (-1e8, torch.float32)):
        steps = torch.randint(0, 5, (3, 3000), generator=g)
        bits = torch.int32 if dtype is torch.float32 else torch.int16
        x = (torch.full((3, 3000), top, dtype=dtype).view(bits) + (steps if top < 0 else -steps).to(bits)).view(dtype)  # so many values lower
        _check(tg, x, torch.tensor([0.1, 0.5, 0.9999]), t * 100 if dtype is torch.float32 and abs(top) == 1e8 else t, None, p, None)


@pytest.mark.parametrize("t", [5e36, 1.5e37, 4e37, 3e38])
@pytest.mark.parametrize("p", [None, 0.2, 0.97])
def test_logits_over_the_whole_range_of_the_type(tg, t, p):
    """Differences that pass the largest float, at temperatures at which they still count."""
    g = torch.Generator().manual_seed(17)
    x = (torch.rand(4, 60007, generator=g, dtype=torch.float64) * 6.8e38 - 3.4e38).float()
    _check(tg, x, torch.tensor([0.0, 0.4, 0.9, 0.9999]), t, None, p, None)
    _check(tg, x, torch.tensor([0.0, 0.4, 0.9, 0.9999]), t, 4000, p, None)
    _check(tg, x, torch.tensor([0.0, 0.4, 0.9, 0.9999]), t, None, p, 0.3)


@pytest.mark.parametrize("t", [1e-45, 1e-30, 0.3, 1.0, 1e3, 1e20, 3e38])
@pytest.mark.parametrize("m", [1e-45, 1e-20, 0.05, 0.7, 0.99999994, 1.0])
def test_least_weights(tg, t, m):
    """At any temperature, of rows all over the type, a little, or around a number far from zero."""
    g = torch.Generator().manual_seed(23)
    y = torch.randn(3, 5000, generator=g)
    for x in (y, y * t, y * 1e30, y + 1e4, y.bfloat16()):
        _check(tg, x, torch.tensor([0.2, 0.55, 0.9999]), t, None, None, m)  # (at 0.5 some rows of weights nearly alike are beyond saying)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("offset", [0, 1, 2, 3, 5, 7])
def test_strides_and_alignment(tg, dtype, offset):
    """Rows that begin anywhere, in a wider matrix whose rest must not count."""
    x, u = _logits(7, 3001, dtype)
    wide = torch.full((7, 3001 + 2 * 8 + offset), math.inf, dtype=dtype, device="cuda")
    view = wide[:, offset:offset + 3001]
    view.copy_(x)
    _check(tg, x, u, 0.8, None, 0.9, device_x=view)
    _check(tg, x, u, 0.8, 30, None, device_x=view)
    _check(tg, x, u, None, None, None, device_x=view)
    one = view[2:3].expand(7, 3001)  # the same row for every u
    _check(tg, x[2:3].expand(7, 3001), u, None, 2500, 0.7, device_x=one)


@pytest.mark.parametrize("dtype", TYPES)
def test_the_largest_vocabulary(tg, dtype):
    """2^18 logits a row, one row of them off every boundary; a top_k as large as integers go."""
    x, u = _logits(3, 2 ** 18, dtype)
    wide = torch.zeros(3, 2 ** 18 + 1, dtype=dtype, device="cuda")
    view = wide[:, 1:]
    view.copy_(x)
    for k, p in ((None, None), (2 ** 63 - 1, None), (None, 0.99), (40000, None), (30, 0.5)):
        _check(tg, x, u, 1.5, k, p, None, device_x=view)


def test_a_row_does_not_depend_on_the_batch(tg):
    """The split over CTAs follows the number of rows; the tokens do not."""
    x, u = _logits(700, 20011, torch.bfloat16)
    x, u = x.cuda(), u.cuda()
    for how in (dict(), dict(top_p=0.9), dict(top_k=4000, top_p=0.99), dict(top_k=40), dict(temperature=5.0, top_p=0.5)):
        whole = tg.sample(x, u, **how)
        for a, b in ((0, 1), (5, 15), (100, 160), (0, 250)):
            assert torch.equal(tg.sample(x[a:b], u[a:b], **how), whole[a:b])


def test_out_streams_graphs(tg):
    x, u = _logits(5, 8000, torch.float16)
    dx, du = x.cuda(), u.cuda()
    want = _check(tg, x, u, 0.9, 50, 0.95)
    out = torch.zeros(5, dtype=torch.int32, device="cuda")
    assert tg.sample(dx, du, 0.9, 50, 0.95, out=out) is out and torch.equal(out, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = tg.sample(dx, du, 0.9, 50, 0.95, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = tg.sample(dx, du, 0.9, 50, 0.95)
    other, v = _logits(5, 8000, torch.float16, seed=9)
    dx.copy_(other)
    du.copy_(v)
    graph.replay()
    assert torch.equal(got, _check(tg, other, v, 0.9, 50, 0.95))
    assert tg.sample(dx[:0], du[:0]).shape == (0,)


def test_refusals(tg):
    x, u = torch.zeros(3, 8, device="cuda"), torch.zeros(3, device="cuda")
    for args, error, says in (((x.long(), u), TypeError, "float16, bfloat16 or float32"), ((x[0], u), ValueError, "rows, vocab"), ((x.cpu(), u), TypeError, "CUDA"),
                              ((x.t(), torch.zeros(8, device="cuda")), ValueError, "contiguous along"), ((x, u[:2]), ValueError, "u must have shape"),
                              ((x, u.double()), TypeError, "float32"), ((x, u, u[:2]), ValueError, "temperature"), ((x, u, 1.0, u), TypeError, "int32"),
                              ((x, u, 1.0, None, u.int()), TypeError, "top_p"), ((x, u, math.nan), tg.TgError, "numbers"),
                              ((x[:, :0], u), tg.TgError, "nothing to draw"), ((torch.zeros(1, 2 ** 18 + 1, device="cuda"), u[:1]), tg.TgError, "vocab")):
        with pytest.raises(error, match=says):
            tg.sample(*args)
    with pytest.raises(ValueError, match="out must have shape"):
        tg.sample(x, u, out=torch.zeros(4, dtype=torch.int32, device="cuda"))
    with pytest.raises(tg.TgError, match="overlaps"):
        tg.sample(x, u, out=u.view(torch.int32))
