"""CPU checks of the entry points around the 8-bit cache: refusals on the host, before anything touches a device,
and the frequency helper."""
import math

import pytest
import torch

from tests import kv_reference as ref

K, V, KS, VS, Q, O = 0x10000000, 0x20000000, 0x30000000, 0x31000000, 0x40000000, 0x50000000
NK, NV, TABLE, LENS, CU, FREQ, WORK = 0x60000000, 0x61000000, 0x70000000, 0x70100000, 0x70200000, 0x70300000, 0x71000000


@pytest.fixture(scope="module")
def tg():
    import __graft_entry__
    __graft_entry__.build()
    import tiled_tensor_core_tcgen05_gb300 as m
    return m


CACHE = dict(k=K, v=V, ks=KS, vs=VS, pages=100, kv_heads=8, page=64, dim=128, fmt=0)
BATCH = dict(table=TABLE, width=16, lens=LENS, cu=CU, batch=4, total=7)
POINTERS = ("k", "v", "ks", "vs", "X", "Y", "pos", "freq", "nk", "nv", "table", "lens", "cu", "q", "qo", "o", "work")


def _args(defaults, changes):
    d = dict(defaults)
    for key, x in changes.items():
        assert key in d, key
        d[key] = x
    return [None if x == 0 and key in POINTERS else x for key, x in d.items()]


ROPE = dict(X=Q, xt=4096, xh=128, Y=O, yt=4096, yh=128, pos=LENS, tokens=7, heads=32, dim=128, freq=FREQ, rotary=128, amp=1.0, layout=0, backward=0, dtype=0, stream=None)
APPEND = dict(CACHE, nk=NK, kt=1024, kh=128, nv=NV, vt=1024, vh=128, **BATCH, max_new=3, freq=FREQ, rotary=128, amp=1.0, layout=0,
              q=Q, qt=4096, qh=128, qo=O, qot=4096, qoh=128, heads=32, dtype=0, stream=None)
READ = dict(CACHE, **BATCH, nk=NK, nv=NV, dtype=0, stream=None)
ATTEND = dict(q=Q, qt=4096, qh=128, o=O, lse=None, **CACHE, **BATCH, heads=32, max_new=3, max_len=1024, causal=1, window=0, scale=0.1, dtype=0,
              work=WORK, work_bytes=1 << 20, stream=None)


@pytest.mark.parametrize("call,defaults,changes,says", [
    ("tg_rope", ROPE, dict(dtype=2), "dtype"),
    ("tg_rope", ROPE, dict(backward=2), "backward"),
    ("tg_rope", ROPE, dict(tokens=-1), "sizes"),
    ("tg_rope", ROPE, dict(dim=2048), "sizes"),
    ("tg_rope", ROPE, dict(xt=-1), "strides of X"),
    ("tg_rope", ROPE, dict(yh=1 << 31), "strides of Y"),
    ("tg_rope", ROPE, dict(layout=2), "layout"),
    ("tg_rope", ROPE, dict(rotary=130), "rotary"),
    ("tg_rope", ROPE, dict(rotary=63), "rotary"),
    ("tg_rope", ROPE, dict(freq=0), "inv_freq"),
    ("tg_rope", ROPE, dict(freq=FREQ + 4), "aligned"),
    ("tg_rope", ROPE, dict(amp=math.inf), "amplitude"),
    ("tg_rope", ROPE, dict(amp=1e39), "amplitude"),
    ("tg_rope", ROPE, dict(X=0), "NULL"),
    ("tg_rope", ROPE, dict(pos=0), "NULL"),
    ("tg_rope", ROPE, dict(Y=O + 1), "aligned"),
    ("tg_rope", ROPE, dict(yh=64), "rows of Y"),
    ("tg_rope", ROPE, dict(yt=1024), "rows of Y"),
    ("tg_rope", ROPE, dict(Y=Q + 256), "overlaps X"),
    ("tg_rope", ROPE, dict(Y=Q, yt=8192), "overlaps X"),
    ("tg_kv_append", APPEND, dict(dtype=-1), "dtype"),
    ("tg_kv_append", APPEND, dict(fmt=2), "format"),
    ("tg_kv_append", APPEND, dict(page=48), "page"),
    ("tg_kv_append", APPEND, dict(dim=96), "head dimensions"),
    ("tg_kv_append", APPEND, dict(pages=-1), "cache sizes"),
    ("tg_kv_append", APPEND, dict(kv_heads=0), "cache sizes"),
    ("tg_kv_append", APPEND, dict(ks=0), "NULL"),
    ("tg_kv_append", APPEND, dict(v=V + 8), "aligned"),
    ("tg_kv_append", APPEND, dict(batch=-1), "sizes"),
    ("tg_kv_append", APPEND, dict(width=1 << 27), "sizes"),
    ("tg_kv_append", APPEND, dict(cu=0), "without cu"),
    ("tg_kv_append", APPEND, dict(max_new=0), "max_new"),
    ("tg_kv_append", APPEND, dict(lens=0), "lens"),
    ("tg_kv_append", APPEND, dict(table=0), "table"),
    ("tg_kv_append", APPEND, dict(lens=LENS + 2), "aligned"),
    ("tg_kv_append", APPEND, dict(kt=-8), "strides of K"),
    ("tg_kv_append", APPEND, dict(rotary=3), "rotary"),
    ("tg_kv_append", APPEND, dict(rotary=0), "Q needs inv_freq"),
    ("tg_kv_append", APPEND, dict(nk=0), "K or V"),
    ("tg_kv_append", APPEND, dict(nv=V), "overlaps K or V"),
    ("tg_kv_append", APPEND, dict(vs=KS + 4), "overlap each other"),
    ("tg_kv_append", APPEND, dict(qo=0), "Q or Q_out"),
    ("tg_kv_append", APPEND, dict(qo=Q + 2), "Q_out overlaps"),
    ("tg_kv_append", APPEND, dict(qo=K), "overlaps the cache"),
    ("tg_kv_append", APPEND, dict(qoh=0), "rows of Q_out"),
    ("tg_kv_read", READ, dict(dtype=5), "dtype"),
    ("tg_kv_read", READ, dict(page=8), "page"),
    ("tg_kv_read", READ, dict(total=1 << 31), "sizes"),
    ("tg_kv_read", READ, dict(nk=0), "K or V"),
    ("tg_kv_read", READ, dict(nv=NV + 2), "aligned"),
    ("tg_kv_read", READ, dict(nv=NK + 16), "overlaps"),
    ("tg_kv_read", READ, dict(nk=VS), "overlaps"),
    ("tg_attention_kv", ATTEND, dict(heads=12), "multiple"),
    ("tg_attention_kv", ATTEND, dict(heads=0), "multiple"),
    ("tg_attention_kv", ATTEND, dict(max_len=-1), "max_len"),
    ("tg_attention_kv", ATTEND, dict(window=-1), "window"),
    ("tg_attention_kv", ATTEND, dict(causal=2), "causal"),
    ("tg_attention_kv", ATTEND, dict(causal=0, window=5), "window needs"),
    ("tg_attention_kv", ATTEND, dict(scale=math.nan), "scale"),
    ("tg_attention_kv", ATTEND, dict(qh=-128), "strides of Q"),
    ("tg_attention_kv", ATTEND, dict(o=O + 2), "aligned"),
    ("tg_attention_kv", ATTEND, dict(o=0), "Q or O"),
    ("tg_attention_kv", ATTEND, dict(o=Q), "overlaps an input"),
    ("tg_attention_kv", ATTEND, dict(lse=O), "overlap each other"),
    ("tg_attention_kv", ATTEND, dict(work=K), "overlaps an input"),
], ids=lambda x: None if isinstance(x, dict) else x)
def test_refused_on_host(tg, call, defaults, changes, says):
    with pytest.raises(tg.TgError) as e:
        getattr(tg, call)(*_args(defaults, changes))
    assert e.value.status == tg.ERR_INVALID_ARG
    assert says in str(e.value)


def test_nothing_to_do_needs_no_device(tg):
    tg.tg_rope(*_args(ROPE, dict(tokens=0)))
    tg.tg_rope(*_args(ROPE, dict(heads=0)))
    tg.tg_kv_append(*_args(APPEND, dict(total=0)))
    tg.tg_kv_append(*_args(APPEND, dict(batch=0, total=0)))
    tg.tg_kv_read(*_args(READ, dict(total=0)))
    tg.tg_attention_kv(*_args(ATTEND, dict(total=0)))
    assert tg.tg_attention_kv_workspace(8, 64, 128, 0, 32, 0, 0, 1, 1024, 0, 0) == 0


def test_binding_refuses_host_tensors_and_types(tg):
    x = torch.zeros(2, 4, 64, dtype=torch.float16)
    with pytest.raises(TypeError, match="CUDA"):
        tg.rope(x, torch.zeros(2, dtype=torch.int32), torch.zeros(32, dtype=torch.float64))
    with pytest.raises(TypeError, match="float8_e4m3fn or int8"):
        tg.KvCache(x, x, x, x)
    c = torch.zeros(2, 1, 16, 64, dtype=torch.int8)
    with pytest.raises(ValueError, match="scales must have shape"):
        tg.KvCache(c, c, torch.zeros(2), torch.zeros(2, 1))
    with pytest.raises(TypeError, match="CUDA"):
        tg.KvCache(c, c, torch.zeros(2, 1), torch.zeros(2, 1))


def test_frequencies(tg):
    f, a = tg.rope_frequencies(128, device="cpu")
    assert a == 1.0 and torch.equal(f, ref.freqs(128))
    g, _ = tg.rope_frequencies(128, scaling="linear", factor=4.0, device="cpu")
    assert torch.equal(g, f / 4)
    g, _ = tg.rope_frequencies(128, scaling="ntk", factor=8.0, device="cpu")
    assert g[0] == f[0] and abs(g[-1] / (f[-1] / 8) - 1) < 1e-12
    g, a = tg.rope_frequencies(128, scaling="yarn", factor=16.0, trained=4096, device="cpu")
    turns = 4096 * f / (2 * math.pi)
    assert torch.equal(g[turns > 40], f[turns > 40]) and torch.allclose(g[turns < 0.9], f[turns < 0.9] / 16, rtol=1e-12)
    assert ((g <= f) & (g >= f / 16 * (1 - 1e-12))).all() and abs(a - (0.1 * math.log(16) + 1)) < 1e-15
    for bad in (dict(rotary=3), dict(rotary=0), dict(rotary=64, scaling="x"), dict(rotary=64, factor=0.5), dict(rotary=2, scaling="ntk", factor=2.0)):
        with pytest.raises(ValueError):
            tg.rope_frequencies(device="cpu", **bad)


def test_reference_gradient_is_the_transpose():
    """The reference's backward rotation against differences of its forward one."""
    g = torch.Generator().manual_seed(3)
    x, dy = (torch.randn(3, 2, 16, generator=g, dtype=torch.float64) for _ in range(2))
    pos, f = torch.tensor([0, 7, 1000]), ref.freqs(8)
    for inter in (False, True):
        dx, _ = ref.rope(dy, pos, f, 1.3, inter, backward=True)
        for at in [(0, 0, 0), (1, 1, 3), (2, 0, 7), (2, 1, 12)]:
            e = torch.zeros_like(x)
            e[at] = 1e-4
            d = (ref.rope(x + e, pos, f, 1.3, inter)[0] - ref.rope(x - e, pos, f, 1.3, inter)[0]) / 2e-4
            assert abs((d * dy).sum() - dx[at]) < 1e-8


# a scale tensor lies on the queries, so that every call is refused on the host, if not for the one reason then for the other
PACKED = dict(q=Q, qo=Q, qt=48 * 128, qot=48 * 128, kt=48 * 128, vt=48 * 128, pages=1, vs=Q)


@pytest.mark.parametrize("changes,meets", [
    (dict(nk=Q + 32 * 256, nv=Q + 40 * 256), False),                                # queries, keys, values
    (dict(nk=Q - 16 * 256, nv=Q - 8 * 256, vs=Q + 6 * 48 * 256), False),                                 # keys and values first
    (dict(nk=Q + 31 * 256, nv=Q + 40 * 256), True),                                 # the last query head is the first key head
    (dict(nk=Q + 32 * 256, nv=Q - 7 * 256, vs=VS), True),
    (dict(nk=Q + 32 * 256 + 2 * 48 * 256, nv=Q + 40 * 256), False),                 # keys of other tokens of the same tensor
    (dict(nk=Q, kt=32 * 128, nv=NV, vs=Q + 236 * 256), True),                               # not slices of one tensor
    (dict(heads=8, qh=384, qoh=384, qt=3200, qot=3200, kt=3200, vt=3200, kh=384, vh=384, nk=Q + 256, nv=Q + 512), False),  # head by head
    (dict(heads=8, qh=384, qoh=384, qt=3200, qot=3200, kt=3200, vt=3200, kh=384, vh=384, nk=Q + 256, nv=Q + 254), True),
    (dict(total=1, nk=Q + 32 * 256, nv=Q + 40 * 256), False),
    (dict(total=1, nk=Q + 32 * 256 - 2, nv=Q + 40 * 256), True),
])
def test_queries_rotated_in_place_beside_keys(tg, changes, meets):
    """The queries are written while keys and values are read: a value in common is refused."""
    args = _args(APPEND, {**PACKED, **changes})
    with pytest.raises(tg.TgError) as e:
        tg.tg_kv_append(*args)
    assert e.value.status == tg.ERR_INVALID_ARG
    assert ("in common" if meets else "Q or Q_out overlaps the cache") in str(e.value)


def test_binding_refuses_tensors_of_another_device(tg):
    """Every tensor of a call goes through this check with the current device."""
    check = tg._binding().check_device
    assert check(0, 0, "Q") is None and check(3, 3, "Q") is None
    with pytest.raises(ValueError, match="Q is on cuda:1, but the current device is cuda:0"):
        check(1, 0, "Q")
