"""GPU checks of attention over a shared prefix where waits run out in both of its passes: the call ends with a timeout that the host
reads, and the next one is what it was before. An arrival a CTA is withheld, and every wait has a limit of 20 ms."""
import pytest
import torch

from tests import test_gpu_kv_large as large
from tests.test_gpu_kv_large import tg  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("counts,lens,groups,shared", [
    ([1, 1], [200, 190], [0, 2], [128]),                                   # few rows a group: the same kernel twice
    ([1, 5, 3, 1], [9000, 9100, 2111, 2200], [0, 2, 4], [8192, 2048]),
    ([1] * 40, [1000 + i for i in range(40)], [0, 40], [960]),             # many: the second pass on tcgen05
    ([2] * 60, [4000 + 7 * i for i in range(60)], [0, 20, 60], [64, 3968]),
])
def test_withheld_arrivals_time_out(tg, counts, lens, groups, shared, dim):  # noqa: F811
    """The workspace holds all ones, so that an entry which no kernel wrote would read as sizes far out of range."""
    cache, table, q = large._made_on_the_gpu(tg, counts, lens, 16, 2, 8, dim, torch.int8, seed=5)
    for g, n in enumerate(shared):
        table[groups[g]:groups[g + 1], :n // 16] = table[groups[g], :n // 16].clone()
    cu, ints = large._ints([0] + torch.tensor(counts).cumsum(0).tolist()), large._ints
    rows = max(sum(counts[a:b]) for a, b in zip(groups, groups[1:]))
    T, H = q.shape[:2]
    lens_d, groups_d, shared_d = ints(lens), ints(groups), ints(shared)
    bounds = dict(max_new=max(counts), max_rows=rows, max_len=max(lens))
    tg.tg_debug_share_always(True)
    try:
        want = tg.attention_kv_shared(q, cache, table, lens_d, groups_d, shared_d, cu, **bounds)
        large._status_ok(tg)
        sizes = (cache.kv_heads, cache.page, dim, cache.fmt)
        need = tg.tg_attention_kv_shared_workspace(*sizes, table.shape[1], H, len(lens), T, len(shared), max(counts), rows, max(lens), tg.FP16)
        work, out = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda"), torch.empty_like(want)
        tg.tg_set_watchdog_ns(20_000_000)
        tg.tg_debug_skip_first_arrive(True)
        try:
            tg.tg_attention_kv_shared(q.data_ptr(), *q.stride()[:2], out.data_ptr(), None, *(t.data_ptr() for t in cache.args), cache.pages, *sizes,
                                      table.data_ptr(), table.shape[1], lens_d.data_ptr(), cu.data_ptr(), len(lens), T, H, max(counts), max(lens), 1,
                                      groups_d.data_ptr(), shared_d.data_ptr(), len(shared), rows, dim ** -0.5, tg.FP16, work.data_ptr(), need,
                                      torch.cuda.current_stream().cuda_stream)
            st, _ = tg.tg_device_status(None)
        finally:
            tg.tg_debug_skip_first_arrive(False)
            tg.tg_set_watchdog_ns(0)
        assert st == tg.ERR_TIMEOUT
        large._status_ok(tg)
        assert torch.equal(tg.attention_kv_shared(q, cache, table, lens_d, groups_d, shared_d, cu, **bounds), want)
        large._status_ok(tg)
    finally:
        tg.tg_debug_share_always(False)
