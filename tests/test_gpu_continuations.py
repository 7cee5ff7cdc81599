"""GPU check of the operators together, as a server uses them to draw several continuations of its prompts: prompts written into the cache,
forked, and step by step tokens drawn, sequences reordered, keys and values appended, the shared prefix attended once; in the
end the pool is compacted and handed to another cache. Every step's attention is checked against the definition in
float64 over what the sequence's own pages hold, and the sequences against a list of tokens kept on the CPU."""
import pytest
import torch

from tests import test_gpu_attention_shared as shared_tests

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


@pytest.mark.parametrize("always", [True, False])
@pytest.mark.parametrize("codes,dtype", [(torch.int8, torch.bfloat16), (torch.float8_e4m3fn, torch.float16)])
def test_continuations(tg, codes, dtype, always):
    g = torch.Generator(device="cuda").manual_seed(5)
    page, kv, heads, dim, vocab, beams = 16, 2, 8, 64, 3000, 5
    prompts = [150, 97]
    cache = tg.KvCache.empty(120, kv, page, dim, dtype=codes)
    made = torch.randn(vocab, kv * 2 + heads, dim, generator=g, device="cuda").to(dtype)  # what the layer makes of a token
    readout = torch.randn(heads * dim, vocab, generator=g, device="cuda") * 0.3
    freq, amplitude = tg.rope_frequencies(dim)

    def step(tokens, table, lens, cu, most):
        x = made[tokens]
        return tg.kv_append(cache, x[:, heads:heads + kv], x[:, heads + kv:], table, lens, cu, max_new=most, Q=x[:, :heads], inv_freq=freq, amplitude=amplitude)

    # prompts: empty sequences get pages, then tokens
    refs, table, lens, spare = tg.kv_fork(cache, torch.zeros(120, dtype=torch.int32, device="cuda"), _ints([[-1] * 16] * 2), _ints([0, 0]), room=150)
    text = [torch.randint(0, vocab, (n,), generator=g, device="cuda") for n in prompts]
    step(torch.cat(text), table, lens, _ints([0, 150, 247]), 150)
    lens = _ints(prompts)
    history = [t.tolist() for t in text]
    parents = [0] * beams + [1] * beams
    groups, shared = _ints([0, beams, 2 * beams]), _ints([n // page * page for n in prompts])
    tokens = None
    try:
        tg.tg_debug_share_always(always)
        for turn in range(24):
            refs, table, lens, spare = tg.kv_fork(cache, refs, table, lens, _ints(parents), room=1)
            assert int(spare) == int((refs == 0).sum()) >= 0
            history = [list(history[p]) for p in parents]
            tokens = [h[-1] for h in history] if tokens is None else [tokens[p] for p in parents]
            q = step(torch.tensor(tokens, device="cuda"), table, lens, None, 1)
            lens = lens + 1
            history = [h + [t] for h, t in zip(history, tokens)]
            o, lse = tg.attention_kv_shared(q, cache, table, lens, groups, shared, max_rows=beams, max_len=240, return_lse=True)
            host = [t.cpu() for t in cache.args]
            shared_tests._check(o, lse, host, table.cpu(), q.cpu(), [1] * 10, lens.tolist(), page, True, dim ** -0.5)
            # the same token after the same text has the same keys, whatever pages it lies in
            logits = o.float().view(10, -1) @ readout
            u = torch.rand(10, generator=g, device="cuda")
            drawn = tg.sample(logits, u, temperature=0.9, top_k=200, top_p=0.95, min_p=0.01)
            assert torch.equal(drawn, torch.stack([tg.sample(logits[i:i + 1], u[i:i + 1], 0.9, 200, 0.95, 0.01)[0] for i in range(10)]))
            tokens = drawn.tolist()
            parents = (torch.randint(0, beams, (2 * beams,), generator=g, device="cuda") + torch.tensor([0] * beams + [beams] * beams, device="cuda")).tolist()
        assert lens.tolist() == [len(h) for h in history]
        # every page is held by the entries that refs says; the text can be read back from the pages of each
        assert torch.equal(torch.bincount(table[table >= 0].long(), minlength=120).int(), refs)
        want, _ = tg.attention_kv_shared(q, cache, table, lens, groups, shared, max_rows=beams, max_len=240, return_lse=True)
        refs, table, moved, used = tg.kv_compact(cache, refs, table)
        assert int(used) == int((refs > 0).sum()) and not (refs[int(used):] > 0).any()
        again, _ = tg.attention_kv_shared(q, cache, table, lens, groups, shared, max_rows=beams, max_len=240, return_lse=True)
        assert torch.equal(again, want)
        other = tg.KvCache.empty(120, kv, page, dim, dtype=codes)
        all_pages = torch.arange(int(used), device="cuda").int()
        tg.kv_copy(cache, all_pages, 119 - all_pages, to=other)
        moved_on, _ = tg.attention_kv_shared(q, other, torch.where(table >= 0, 119 - table, -1), lens, groups, shared, max_rows=beams, max_len=240, return_lse=True)
        assert torch.equal(moved_on, want)
        refs, table, lens, spare = tg.kv_fork(cache, refs, table, lens, _ints([-1] * 3))
        assert int(spare) == 120 and not refs.any() and lens.tolist() == [0] * 3
    finally:
        tg.tg_debug_share_always(False)
    st, where = tg.tg_device_status(None)
    assert st == tg.OK, f"device status {st} at {where}"


@pytest.mark.parametrize("codes", [torch.int8, torch.float8_e4m3fn])
def test_forked_texts_hold_what_they_say(tg, codes):
    """After many forks and appends each sequence's keys are those of its own text (values are tokens' numbers, exact in the cache)."""
    g = torch.Generator().manual_seed(8)
    page, n = 16, 7
    cache = tg.KvCache.empty(80, 1, page, 64, dtype=codes)
    refs, table, lens, _ = tg.kv_fork(cache, torch.zeros(80, dtype=torch.int32, device="cuda"), _ints([[-1] * 10] * n), _ints([0] * n), room=1)
    text = [[] for _ in range(n)]
    for turn in range(60):
        tokens = torch.randint(1, 8, (n,), generator=g)
        k = torch.zeros(n, 1, 64, dtype=torch.float16)
        k[:, 0, 0] = 7.0  # the scale of every page is the same
        k[:, 0, 1] = tokens.half()
        tg.kv_append(cache, k.cuda(), k.cuda(), table, lens)
        lens = lens + 1
        text = [t + [int(x)] for t, x in zip(text, tokens)]
        parents = torch.randint(0, n, (n,), generator=g).tolist()
        refs, table, lens, spare = tg.kv_fork(cache, refs, table, lens, _ints(parents), room=1)
        text = [list(text[p]) for p in parents]
    cu = [0]
    for t in text:
        cu.append(cu[-1] + len(t))
    K, V = tg.kv_read(cache, table, _ints([0] * n), _ints(cu), cu[-1])
    got = K[:, 0, 1].float().cpu()
    tol = 7.0 / 127 / 2 + 2.0 ** -8 if codes is torch.int8 else 7.0 * 2.0 ** -4  # half a code, and the read's rounding; half a step of e4m3
    assert ((got - torch.tensor(sum(text, [])).float()).abs() <= tol).all()
    assert int(spare) >= 0
