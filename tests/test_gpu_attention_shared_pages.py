"""GPU checks of attention over a shared prefix of which pages are missing, in what is shared and in the sequences' own parts: reported, their keys left
out, the others seen."""
import pytest
import torch

from tests import kv_reference as ref
from tests import test_gpu_attention_kv as attend
from tests.test_gpu_attention_kv import _ints, _status_ok, tg  # noqa: F401
from tests.test_gpu_attention_shared import always  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page,dim", [(16, 64), (64, 128), (128, 64)])
@pytest.mark.parametrize("batch", [3, 40])   # few rows a group, and many
def test_pages_that_are_missing(tg, page, dim, batch):  # noqa: F811
    n, lens = 1024, [1024 + page + 7 + 3 * (i % 5) + (1 if page > 32 else 0) for i in range(batch)]
    cache, host, table, q = attend._case(tg, [1] * batch, lens, page, 2, 4, dim, 0, 0, seed=page)
    slots = n // page
    table[:, :slots] = table[0, :slots]
    pages = host[0].shape[0]
    bad = table.clone()
    gone = sorted({0, slots // 2, slots - 1})
    bad[:, gone] = torch.tensor([-1, 2 ** 31 - 1, pages], dtype=torch.int32)[:len(gone)]
    bad[1, slots] = -2 ** 31                             # the first of its own
    out, lse = tg.attention_kv_shared(q.cuda(), cache, bad.cuda(), _ints(lens), _ints([0, batch]), _ints([n]), max_len=max(lens), return_lse=True)
    assert tg.tg_device_status(None)[0] == tg.ERR_BOUNDS
    for i in (0, 1, 2, batch - 1):
        seen = [s for s in range(-(-lens[i] // page)) if s not in gone and not (i == 1 and s == slots)]
        k, v = (torch.cat([ref.gather(c, s, table[i, [j]].long(), min(page, lens[i] - j * page)) for j in seen]) for c, s in ((host[0], host[2]), (host[1], host[3])))
        o, want, tol, ltol = ref.attention(q[i:i + 1].double(), k, v, len(k), False, 0, dim ** -0.5)
        ref.near(out[i:i + 1], o, tol + 2.0 ** -19 * v.abs().max() + o.abs() * ref.half_step(out.dtype) + 2.0 ** -25, f"sequence {i}")
        ref.near(lse[i:i + 1], want, ltol + 2.0 ** -19, f"lse of sequence {i}")
    _status_ok(tg)
    bad[:, :slots] = -1                                  # nothing of what is shared is there
    out, lse = tg.attention_kv_shared(q.cuda(), cache, bad.cuda(), _ints(lens), _ints([0, batch]), _ints([n]), max_len=max(lens), return_lse=True)
    assert tg.tg_device_status(None)[0] == tg.ERR_BOUNDS
    own = tg.attention_kv(q.cuda(), cache, bad[:, slots:].contiguous().cuda(), _ints([x - n for x in lens]), max_len=max(lens), return_lse=True)
    tg.tg_device_status(None)
    # both round each weight by 2^-11 of itself, and the result by half a step
    most = (host[1].double() * host[3].double()[:, :, None, None]).nan_to_num(0.0).abs().max()
    ref.near(out, own[0].double().cpu(), own[0].abs().double().cpu() * 2 * ref.half_step(out.dtype) + 2.0 ** -10 * most)
    ref.near(lse, own[1].double().cpu(), torch.full_like(lse, 2.0 ** -18).double().cpu())
