"""GPU checks of which sequences of a group share its prefix: those with at least as many tokens before their new ones as are shared, be
that a whole number of 64 or not. A sequence one token short has pages of its own, and is attended over them."""
import pytest
import torch

from tests import test_gpu_attention_kv as attend
from tests import test_gpu_attention_shared as shared_tests
from tests.test_gpu_attention_kv import _ints, _status_ok, tg  # noqa: F401
from tests.test_gpu_attention_shared import always  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page,dim,share", [(16, 64, 4), (64, 128, 4), (128, 128, 1), (16, 128, 16)])
@pytest.mark.parametrize("n", [65, 100, 127, 128, 129, 700])
@pytest.mark.parametrize("most", [1, 3])
def test_one_token_short_is_a_sequence_of_its_own(tg, page, dim, share, n, most):  # noqa: F811
    """Tokens before the new ones: on both sides of what is shared, and of the whole number of 64 below it. The first of the group is a short one."""
    held = [n // 64 * 64, n, n - 1, n + 1, n // 64 * 64 - 1, n // 64 * 64 + 1, 2 * n, 0, n, n - 1]
    for group in ([0, 10], [0, 3, 10], [2, 4], [2, 3, 9]):
        counts = [1 + i % most for i in range(10)]
        lens = [h + c for h, c in zip(held, counts)]
        cache, host, table, q = attend._case(tg, counts, lens, page, 2, share, dim, 0, 0, seed=n)
        shared, m = [n] * (len(group) - 1), -(-n // page)
        for a, b in zip(group, group[1:]):  # those that hold what is shared have the longest one's pages for it
            members = [i for i in range(a, b) if held[i] >= n]
            for i in members:
                table[i, :m] = table[max(members, key=lambda j: lens[j]), :m]
        cu = [0] + torch.tensor(counts).cumsum(0).tolist()
        rows = max(cu[b] - cu[a] for a, b in zip(group, group[1:]))
        for causal in (True, False):
            out, lse = tg.attention_kv_shared(q.cuda(), cache, table.cuda(), _ints(lens), _ints(group), _ints(shared), _ints(cu), max_new=max(counts), max_rows=rows,
                                              causal=causal, return_lse=True)
            shared_tests._check(out, lse, host, table, q, counts, lens, page, causal, dim ** -0.5)
    _status_ok(tg)
