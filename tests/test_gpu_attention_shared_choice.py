"""GPU checks of when attention over a shared prefix takes a pass of its own for what is shared: where by the bounds of the
call it can save 256 MB of reading. Which way a call goes shows in the workspace that it asks for; without that pass it is
attention_kv to the bit, with it what the same call gives when the pass is asked for, and within the definition's tolerance."""
import pytest
import torch

from tests import test_gpu_attention_kv as attend
from tests import test_gpu_attention_shared as shared_tests
from tests.test_gpu_attention_kv import _ints, _status_ok, tg  # noqa: F401

pytestmark = pytest.mark.gpu
KV, SHARE, DIM, PAGE = 2, 4, 128, 64
BORDER = 2 ** 28 // (KV * DIM * 2)  # tokens whose keys and values are 256 MB


@pytest.mark.parametrize("batch,groups,max_rows,most,max_len,width,pays", [
    (65, [0, 65], 65, 1, BORDER // 64, 128, True),            # 64 sequences spared
    (65, [0, 65], 65, 1, BORDER // 64 - 1, 128, False),
    (64, [0, 64], 64, 1, BORDER // 64, 128, False),
    (65, [0, 65], 65, 1, BORDER // 64, 127, False),           # the table is the bound
    (65, [0, 65], 65, 1, 10 * BORDER, 128, True),
    (130, [1, 34, 67], 33, 1, BORDER // 64, 128, True),       # two groups, and as many sequences in none
    (130, [1, 34, 67], 33, 1, BORDER // 64 - 1, 128, False),
    (65, [3, 5], 2, 1, BORDER // 64, 128, False),             # a group of two spares one
    (65, [3, 5], 2, 1, BORDER, 8192, True),
    (65, [3, 5], 2, 1, BORDER - 1, 8192, False),
    (65, [3, 5], None, 1, BORDER // 64, 128, True),           # a bound left to the call is taken for a large group
    (65, [0] * 33 + [65], 65, 1, BORDER // 32, 256, True),    # all but one group without sequences: no more than sequences less groups
    (65, [0] * 33 + [65], 65, 1, BORDER // 32 - 1, 256, False),
    (65, [0, 65], 65, 17, 10 * BORDER, 8192, False),          # 68 rows of a sequence and kv head
])
def test_which_way_a_call_goes(tg, batch, groups, max_rows, most, max_len, width, pays):  # noqa: F811
    counts, lens, n = [1] * batch, [300 + 5 * (i % 9) for i in range(batch)], 256
    cache, host, table, q = attend._case(tg, counts, lens, PAGE, KV, SHARE, DIM, 0, 0, seed=batch)
    shared = [n if a < b else 0 for a, b in zip(groups, groups[1:])]
    shared_tests._share(table, groups, shared, lens, PAGE)
    wide = torch.full((batch, width), -1, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    args, bounds = (q.cuda(), cache, wide.cuda(), _ints(lens)), dict(max_new=most, max_len=max_len, return_lse=True)
    cu = _ints(list(range(batch + 1))) if most > 1 else None
    sizes = (KV, PAGE, DIM, cache.fmt)
    alone = tg.tg_attention_kv_workspace(*sizes, KV * SHARE, batch, batch, most, max_len, 0, tg.FP16)
    asked = tg.tg_attention_kv_shared_workspace(*sizes, width, KV * SHARE, batch, batch, len(shared), most, max_rows or batch, max_len, tg.FP16)
    assert (asked > alone) if pays else (asked == alone)
    out, lse = tg.attention_kv_shared(*args, _ints(groups), _ints(shared), cu, max_rows=max_rows, **bounds)
    if pays:
        tg.tg_debug_share_always(True)
        try:
            want = tg.attention_kv_shared(*args, _ints(groups), _ints(shared), cu, max_rows=max_rows, **bounds)
        finally:
            tg.tg_debug_share_always(False)
    else:
        want = tg.attention_kv(*args, cu, **bounds)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    shared_tests._check(out, lse, host, wide, q, counts, lens, PAGE, True, DIM ** -0.5)
    _status_ok(tg)
