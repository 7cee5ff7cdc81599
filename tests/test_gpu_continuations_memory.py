"""GPU check that the entry points around continuations of one prompt allocate nothing: the device's free memory is the same after as before, over
calls of several sizes through the C ABI with the caller's workspaces."""
import pytest
import torch

from tests.test_gpu_kv_pages import _cache, _ints, _status, tg  # noqa: F401

pytestmark = pytest.mark.gpu


def test_no_device_memory_is_taken(tg):  # noqa: F811
    kv, page, dim, heads = 2, 64, 128, 16
    stream = torch.cuda.current_stream().cuda_stream
    calls = []
    for pages, batch, width in ((40, 3, 9), (3000, 100, 200)):
        cache, other = _cache(tg, pages, kv, page, dim), _cache(tg, pages, kv, page, dim, seed=1)
        at = [t.data_ptr() for t in cache.args]
        sizes = (kv, page, dim, cache.fmt)
        refs, table, lens = _ints([1] * 5 + [0] * (pages - 5)), torch.full((batch, width), -1, dtype=torch.int32, device="cuda"), _ints([300] + [0] * (batch - 1))
        table[0, :5] = _ints([0, 1, 2, 3, 4])
        parents, src, dst = _ints([0] * batch), _ints([0, 1, 2]), _ints([9, 7, 5])
        refs_out, table_out, lens_out, one, moved = (torch.empty_like(t) for t in (refs, table, lens, _ints([0]), refs))
        need = max(tg.tg_kv_fork_workspace(pages, page, batch, batch, width), tg.tg_kv_compact_workspace(pages),
                   tg.tg_attention_kv_shared_workspace(*sizes, width, heads, batch, batch, 1, 1, batch, width * page, tg.FP16))
        work = torch.empty(need, dtype=torch.uint8, device="cuda")
        q = torch.randn(batch, heads, dim, device="cuda").half()
        o, full = torch.empty_like(q), table[:1].expand(batch, width).contiguous()
        groups, shared, long = _ints([0, batch]), _ints([256]), _ints([300] * batch)
        x, u, tokens = torch.randn(batch, 50000, device="cuda"), torch.rand(batch, device="cuda"), torch.empty(batch, dtype=torch.int32, device="cuda")
        keep = (cache, other, refs, table, lens, parents, src, dst, refs_out, table_out, lens_out, one, moved, work, q, o, full, groups, shared, long, x, u, tokens)

        def run(at=at, to=[t.data_ptr() for t in other.args], sizes=sizes, pages=pages, batch=batch, width=width, need=need, p=[t.data_ptr() for t in keep[2:]], keep=keep):
            refs, table, lens, parents, src, dst, refs_out, table_out, lens_out, one, moved, work, q, o, full, groups, shared, long, x, u, tokens = p
            tg.tg_kv_copy(*at, pages, *to, pages, *sizes, src, dst, 3, stream)
            tg.tg_kv_fork(*at, pages, *sizes, refs, table, width, lens, batch, parents, batch, 1, refs_out, table_out, lens_out, one, work, need, stream)
            tg.tg_kv_compact(*at, pages, *sizes, refs, table, width, batch, refs_out, table_out, moved, one, work, need, stream)
            tg.tg_attention_kv_shared(q, heads * dim, dim, o, None, *at, pages, *sizes, full, width, long, None, batch, batch, heads, 1, width * page, 1, groups, shared, 1, batch,
                                      0.1, tg.FP16, work, need, stream)
            for k, top_p in ((0, 1.0), (50, 1.0), (0, 0.9)):
                tg.tg_sample(x, 50000, batch, 50000, tg.FP32, u, None, 1.0, None, k, None, top_p, None, 0.0, tokens, stream)
        calls.append(run)
    for run in calls:  # kernels are loaded
        run()
    torch.cuda.synchronize()
    before = torch.cuda.mem_get_info()[0]
    for run in calls + calls[::-1]:
        run()
    torch.cuda.synchronize()
    assert torch.cuda.mem_get_info()[0] == before
    _status(tg)
