"""The operators around the paged 8-bit cache from their definitions, in float64 on the CPU, and how far a
correct result may be from them. Half a step of rounding is torch.finfo(t).eps / 2 of the value."""
import math

import torch

QMAX = {torch.float8_e4m3fn: 448.0, torch.int8: 127.0}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def freqs(rotary, base=10000.0):
    return base ** (-torch.arange(0, rotary, 2, dtype=torch.float64) / rotary)


def rope(x, pos, freq, amplitude, interleaved, backward=False):
    """(values, size): size bounds the products' terms, amplitude * (|a| + |b|) of each pair."""
    x = x.double()
    n = 2 * freq.numel()
    a, b = (slice(0, n, 2), slice(1, n, 2)) if interleaved else (slice(0, n // 2), slice(n // 2, n))
    t = pos.double()[:, None] * freq
    c, s = t.cos()[:, None] * amplitude, t.sin()[:, None] * (-amplitude if backward else amplitude)
    y, size = x.clone(), torch.zeros_like(x)
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    size[..., a] = size[..., b] = (x[..., a].abs() + x[..., b].abs()) * abs(amplitude)
    return y, size


def code_step(u, dtype):
    """The spacing of the codes around u (in units of the scale)."""
    if dtype is torch.int8:
        return torch.ones_like(u)
    _, e = torch.frexp(u)
    return torch.ldexp(torch.ones_like(u), torch.where(u == 0, -6, (e - 1).clamp(min=-6)) - 3)


def append(k, codes, scales, table, lens, counts, page, dtype):
    """What appending rows k (total, heads, dim; float64) leaves: (units, scales, written): codes before their
    rounding (held codes of a page whose scale grew, times old / new scale), the scales, and which codes the
    call may change."""
    units = codes.double().clone()
    scales = scales.double().clone()
    written = torch.zeros(units.shape, dtype=torch.bool)
    row = 0
    for i, n in enumerate(counts):
        at, end = lens[i], lens[i] + n
        while at < end:
            many = min(page - at % page, end - at)
            p, o = int(table[i, at // page]), at % page
            x = k[row:row + many]
            finite = torch.where(x.isfinite(), x.abs(), 0.0)
            most = finite.amax((0, 2))
            s = (most / QMAX[dtype]).clamp(min=2.0 ** -60)
            if o:
                s = torch.maximum(s, scales[p])
                units[p, :, :o] *= (scales[p] / s)[:, None, None]
                written[p, :, :o] = True
            x = torch.where(x.isinf(), torch.sign(x) * most[:, None], x)
            units[p, :, o:o + many] = (x / s[:, None]).transpose(0, 1)
            written[p, :, o:o + many] = True
            scales[p] = s
            at, row = at + many, row + many
    return units, scales, written


def gather(codes, scales, pages, n):
    """(n, heads, dim) float64 of a sequence's first n tokens."""
    x = codes.view(torch.uint8)[pages].view(codes.dtype).double() * scales.double()[pages][:, :, None, None]
    return x.permute(0, 2, 1, 3).reshape(-1, codes.shape[1], codes.shape[3])[:n]


def attention(q, k, v, length, causal, window, scale):
    """One sequence: q (n, heads, dim), k and v (length, kv, dim), float64. (o, lse, tolerance of o before its own
    rounding, tolerance of lse).

    The weights come from scores whose dot products add dim terms in 32 bits (an error of at most dim * 2^-24 of
    the sum of |q k|, doubled for the tensor core's own order and for the factors applied to them), through a 2^x
    good to 2^-21, rounded to 16 bits (2^-11) for their product with the values, which adds `length` terms in 32
    bits; weights under 2^-14 of the largest are rounded in steps of 2^-24 of it."""
    n, heads, dim = q.shape
    share = heads // k.shape[1]
    pos = torch.arange(length - n, length)[:, None]
    j = torch.arange(length)
    seen = (j <= pos) if causal else torch.ones(n, length, dtype=torch.bool)
    if window:
        seen = seen & (j > pos - window)
    o, tol = torch.zeros(n, heads, dim, dtype=torch.float64), torch.zeros(n, heads, dim, dtype=torch.float64)
    lse, lse_tol = torch.full((n, heads), -math.inf, dtype=torch.float64), torch.zeros(n, heads, dtype=torch.float64)
    if length == 0:
        return o, lse, tol, lse_tol
    some = seen.any(1)
    for h in range(heads):
        kh, vh = k[:, h // share], v[:, h // share]
        z = (q[:, h] @ kh.T * scale).masked_fill(~seen, -math.inf)
        size = (q[:, h].abs() @ kh.abs().T * abs(scale)).masked_fill(~seen, 0.0).amax(1)
        ds = 2 * dim * 2.0 ** -24 * size + 2.0 ** -21
        l = torch.logsumexp(z, 1)
        p = (z - l[:, None]).exp().nan_to_num(0.0)
        o[some, h] = (p @ vh)[some]
        most = torch.where(seen[:, :, None], vh.abs()[None], 0.0).amax(1) if n * length * dim < 1 << 24 else vh.abs().amax(0).expand(n, -1)
        small = 2.0 ** -25 * seen.sum(1)[:, None] * most
        tol[:, h] = (2 * ds + 2.0 ** -11 + length * 2.0 ** -24)[:, None] * (p @ vh.abs()) + small
        lse[:, h] = torch.where(some, l, -math.inf)
        lse_tol[:, h] = ds + length * 2.0 ** -24 + 2.0 ** -21 * (1 + l.abs().nan_to_num(0.0, 0.0, 0.0))
    return o, lse, tol, lse_tol


def near(got, want, tol, what=""):
    """Same infinities and NaN; elsewhere within tol."""
    got, want = got.double().cpu(), want.double()
    assert got.shape == want.shape, what
    fine = want.isfinite()
    assert torch.equal(got.isnan(), want.isnan()), f"{what}: NaN elsewhere"
    assert torch.equal(got[~fine & ~want.isnan()], want[~fine & ~want.isnan()]), f"{what}: infinities elsewhere"
    off = ((got - want).abs() - tol)[fine]
    assert not off.numel() or off.max() <= 0, f"{what}: {int((off > 0).sum())} of {off.numel()} out of tolerance, by up to {off.max():.3g}"
