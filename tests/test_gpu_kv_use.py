"""GPU checks of how the cache operators' tensor forms treat what a program does around them."""
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
