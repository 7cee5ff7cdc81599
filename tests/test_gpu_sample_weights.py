"""GPU checks of how exactly logits are weighed, of logits near zero and far from it by their temperature. A row's weights are right to 2^-37 of
themselves, so the border between the tokens of a row of two is right to 2^-36 of the sum; u has steps of 2^-24 there, and rows are left out
whose u lies nearer than 2^-34 to the border. Equal logits have equal weights, exactly, wherever they are."""
import math

import pytest
import torch

from tests import test_gpu_sample as sample_tests
from tests.test_gpu_sample import tg  # noqa: F401

pytestmark = pytest.mark.gpu
FAR = [0.3, 3.0, 7.0, 12.0, 20.0, 40.0, 63.0, 70.0, 100.0, 127.0, 150.0, 199.0, 250.0, 1000.0]  # the largest logit, in temperatures


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("far", FAR)
@pytest.mark.parametrize("cut", [False, True])
def test_border_of_two_tokens(tg, far, sign, cut):  # noqa: F811
    """The float of u next to the border and its neighbours: below it the first token, from it on the second. With `cut` the same border
    decides whether top_p keeps the less likely one."""
    n = 20000
    g = torch.Generator().manual_seed(int(far * 10) + (sign > 0))
    t = torch.exp(torch.rand(n, generator=g) * 4 - 2)
    a = sign * far * t * (1 + torch.rand(n, generator=g) / 16)
    b = a - t * torch.rand(n, generator=g) * 3
    x = torch.stack([a, b], 1)
    if not cut:
        flip = torch.rand(n, generator=g) < 0.5
        x = torch.where(flip[:, None], x.flip(1), x)
    y = x.double() / t.double()[:, None]
    border = torch.sigmoid(y[:, 0] - y[:, 1])  # the first one's share
    for step in (-1, 0, 1):
        u = border.float()
        if step:
            u = torch.nextafter(u, torch.tensor(math.inf * step))
        sure = ((u.double() - border).abs() > sample_tests.NEAR) & (u < 1)
        assert sure.sum() > n * 0.9
        if cut:  # the second one is kept, and drawn by the largest u, where the first has less than top_p
            got = tg.sample(x.cuda(), torch.full((n,), 0.99999994, device="cuda"), temperature=t.cuda(), top_p=u.cuda()).cpu()
            want = (u.double() > border).int()
        else:
            got = tg.sample(x.cuda(), u.cuda(), temperature=t.cuda()).cpu()
            want = (u.double() >= border).int()
        wrong = (got != want) & sure
        assert not wrong.any(), f"{int(wrong.sum())} of {n}, as at x {x[wrong][0].tolist()}, T {float(t[wrong][0])}, u {float(u[wrong][0])}: {int(got[wrong][0])}"


@pytest.mark.parametrize("far", FAR)
@pytest.mark.parametrize("dtype", sample_tests.TYPES)
def test_equal_logits_far_from_zero(tg, far, dtype):  # noqa: F811
    """A row whose largest logits are alike, among others far below: what is kept is counted, exactly."""
    g = torch.Generator().manual_seed(int(far))
    for t, vocab in ((1.0, 5003), (0.7, 40000), (90.98, 30001)):
        for sign in (1.0, -1.0):
            top = torch.tensor(sign * far * t).to(dtype)
            if not top.isfinite():
                continue
            x = torch.where(torch.rand(4, vocab, generator=g) < 0.3, top.float(), top.float() - 60 * t - 60 * abs(float(top)) * 2.0 ** -8).to(dtype)
            for k, p in ((None, None), (None, 0.5), (2048, 0.5), (2048, None), (100, 0.25), (1000, 0.75)):
                sample_tests._check(tg, x, torch.tensor([0.0, 0.45756954, 0.75, 0.99999994]), t, k, p, None)


@pytest.mark.parametrize("dtype", sample_tests.TYPES)
@pytest.mark.parametrize("far", [10.0, 60.0, 120.0, 190.0])
def test_rows_far_from_zero(tg, far, dtype):  # noqa: F811
    """Ordinary spreads around a number far from zero by the temperature."""
    for vocab in (300, 9001, 131071):
        x, u = sample_tests._logits(6, vocab, torch.float32, 1.0 if dtype is torch.float32 else 4.0)
        for t in (0.25, 1.0):
            for sign in (1, -1):
                y = (x * t + sign * far * t).to(dtype)
                for k, p, m in ((None, None, None), (None, 0.9, None), (50, None, None), (3000, 0.95, None), (None, None, 0.02), (40, 0.8, 0.01)):
                    got = tg.sample(y.cuda(), u.cuda(), t, k, p, m).tolist()
                    for i in range(6):
                        want, sure = sample_tests.draw(y[i], float(u[i]), t, k or 0, 1.0 if p is None else float(torch.tensor(p)), 0.0 if m is None else float(torch.tensor(m)))
                        assert not sure or got[i] == want, (i, vocab, t, sign, k, p, m)


@pytest.mark.parametrize("dtype", sample_tests.TYPES)
@pytest.mark.parametrize("vocab", [50, 3001, 30000, 131072])
def test_numbers_next_to_the_borders_of_longer_rows(tg, dtype, vocab):  # noqa: F811
    """top_p is the float at, or next to, a token's edge in falling order; u the one at an edge of what that keeps, by index."""
    g = torch.Generator().manual_seed(vocab)
    for t, spread, around, k, m in ((1.0, 2.5, 0.0, 0, 0.0), (0.75, 1.0, 20.0, 0, 0.0), (2.0, 0.5, -150.0, 0, 1e-4), (1.0, 2.5, 90.0, 2500, 0.0), (1.0, 6.0, 0.0, 40, 0.05)):
        rows = 6
        x = ((torch.randn(rows, vocab, generator=g) * spread + around) * t).to(dtype)
        u, p = torch.empty(rows), torch.ones(rows)
        for i in range(rows):
            y, at = ((x[i].double() - float(x[i].max())) / t).sort(descending=True, stable=True)
            w = y.exp() * (y > -43 * math.log(2))
            if k:
                w[k:] = 0
            if m:
                w *= y >= math.log(float(torch.tensor(m)))
            some = torch.rand(2, generator=g).tolist()
            toward = torch.tensor([2.0, -1.0])[i % 2]
            if i % 3:
                edge = (w.cumsum(0) / w.sum())[int((w.cumsum(0) > some[0] * w.sum()).nonzero()[0])].float()
                p[i] = min(edge if i % 3 == 1 else torch.nextafter(edge, toward), torch.tensor(1.0))
                w = w * (w.cumsum(0) - w < float(p[i]) * w.sum())
            c = torch.zeros_like(w).scatter_(0, at, w).cumsum(0)
            edge = (c[int((c > some[1] * c[-1]).nonzero()[0])] / c[-1]).float()
            u[i] = edge if i == 0 else torch.nextafter(edge, toward)
        got = tg.sample(x.cuda(), u.cuda(), t, k, p.cuda(), m).tolist()
        for i in range(rows):
            want, sure = sample_tests.draw(x[i], float(u[i]), t, k, float(p[i]), float(torch.tensor(m)))
            assert not sure or got[i] == want, (i, t, around, k, m, float(p[i]), float(u[i]))
