"""What is measured of the operators around attention over a cache held in 8 bits: rotary positions, writing new keys and values
into the cache (quantised as they are written, optionally rotated on the way), reading the cache back, and attention over it.

The cache is paged. A page holds `page` consecutive tokens of one sequence, head by head: codes of shape (pages, kv_heads, page,
head_dim) in e4m3 or int8, and one float32 scale for each (page, kv_head); a value is code * scale. A sequence's pages are the
entries of its row of `table` in order. Packed tensors hold the sequences' new tokens one after another, sequence i's in rows
cu[i] .. cu[i + 1] - 1.

The plain forms below are elementary torch operations in 32 bits (rotation angles in 64).
"""
import math
import random

import torch

own = False

FLOOR = 2.0 ** -60  # the least scale of a block: a block of zeros has this one
QMAX = {"e4m3": 448.0, "int8": 127.0}
STORE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
HALF = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a single sequence's decode step: queries and keys of one token, where the call's latency is all there is
        _rope("rope_one_token", tokens=1, heads=40, slots=48, far=4095),
        # a long prompt's queries and keys, rotated where the fused projection left them (48 head slots a token, values after
        # them); long-context scaling by frequency bands, positions far beyond the trained length
        _rope("rope_prompt_far", tokens=8192, heads=40, slots=48, far=1000000, scaling="yarn", factor=16.0),
        # training: gradient through a rotation of half of each head in the interleaved layout, an odd number of tokens
        _rope("rope_part_gradient", tokens=4099, heads=32, slots=32, rotary=64, layout="interleaved", dtype="bf16", backward=True),
        # a decode step of a full batch: one token a sequence, keys rotated, queries with them, into partly filled pages
        _append("append_decode_rotated", batch=256, longest=4096, most=1, rotate=True, dtype="bf16", mix=1),
        # prompts of several lengths quantised at once into pages of 32 tokens
        _append("append_prompts_int8", batch=7, longest=5000, most=4500, store="int8", page=32, mix=2),
        # a few sequences' cached blocks read back, odd lengths
        _read("read_ragged_int8", batch=5, longest=777, store="int8", page=16, head_dim=64, kv_heads=4, mix=3),
        # a long cache read back, to hand it to another process or to attend in full precision
        _read("read_long", batch=16, longest=16384, dtype="bf16", mix=4),
        # one sequence's decode step over a short cache: latency
        _attend("attend_one_short", batch=1, longest=1023),
        # a decode step of a full batch of ragged lengths, a few of its slots idle
        _attend("attend_decode_ragged", batch=64, longest=8192, idle=3, mix=5),
        # few sequences with very long caches, split over the whole GPU
        _attend("attend_decode_long", batch=4, longest=131071, store="int8", page=128, lse=True, mix=6),
        # verification of a few drafted tokens a sequence, seven query heads a key head, heads of 64, small pages, a window
        _attend("attend_drafts_window", batch=33, longest=6000, most=5, heads=28, kv_heads=4, head_dim=64, page=16,
                dtype="bf16", window=2048, mix=7),
        # prompt chunks against their caches: the products count
        _attend("attend_chunks", batch=2, longest=8192, most=4096, mix=8),
    ]


def draw(rng):
    kind = rng.choice(["rope", "append", "append", "read", "attend", "attend", "attend"])
    dtype, store, page = rng.choice(["fp16", "bf16"]), rng.choice(["e4m3", "int8"]), rng.choice([16, 32, 64, 128])
    dim, kv = rng.choice([64, 128, 128]), rng.choice([1, 2, 4, 8])
    share, mix = rng.choice([1, 2, 3, 4, 5, 7, 8]), rng.randrange(1 << 20)
    if kind == "rope":
        heads = rng.randint(1, 40)
        case = _rope(None, tokens=_log(rng, 1, 8192), heads=heads, slots=heads + rng.choice([0, 8]), far=_log(rng, 1, 1 << 21), head_dim=dim,
                     rotary=rng.choice([dim, dim, dim // 2, dim - 16]), layout=rng.choice(["half", "interleaved"]), dtype=dtype,
                     scaling=rng.choice(["none", "linear", "ntk", "yarn"]), factor=rng.choice([2.0, 4.0, 8.0, 32.0]), backward=rng.random() < 0.3)
    elif kind == "append":
        batch = _log(rng, 1, 256)
        most = 1 if rng.random() < 0.4 else _log(rng, 1, max(1, 16384 // batch))
        rotate = rng.random() < 0.5
        # codes of rotated keys are compared as the e4m3 values they are; whole numbers would have to agree where sines do not
        case = _append(None, batch=batch, longest=most + _log(rng, 1, 4096), most=most, rotate=rotate, layout=rng.choice(["half", "interleaved"]),
                       store="e4m3" if rotate else store, page=page, heads=kv * share, kv_heads=kv, head_dim=dim, dtype=dtype, mix=mix)
    elif kind == "read":
        batch = _log(rng, 1, 64)
        case = _read(None, batch=batch, longest=_log(rng, 1, 131072 // batch), store=store, page=page, kv_heads=kv, head_dim=dim, dtype=dtype, mix=mix)
    else:
        batch = _log(rng, 1, 128)
        shape = rng.choice(["decode", "decode", "drafts", "chunk"])
        if shape == "chunk":
            batch = rng.randint(1, 3)
            most = _log(rng, 17, 4096 // batch)
            longest = most + _log(rng, 1, 4096)
            kv, share = min(kv, 4), min(share, 4)
        else:
            most = 1 if shape == "decode" else rng.randint(2, 16)
            longest = most + _log(rng, 1, 262144 // batch)
        window = _log(rng, 16, longest) if longest > 64 and rng.random() < 0.25 else 0
        case = _attend(None, batch=batch, longest=longest, most=most, heads=kv * share, kv_heads=kv, head_dim=dim, store=store, page=page, dtype=dtype,
                       window=window, idle=1 if batch > 4 and rng.random() < 0.3 else 0, lse=rng.random() < 0.3, mix=mix)
    case.pop("name")
    return case


def _log(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.49)))))))


def _rope(name, tokens, heads, slots, far=8192, head_dim=128, rotary=None, layout="half", dtype="fp16", scaling="none", factor=1.0, backward=False):
    return {"name": name, "op": "rope", "tokens": tokens, "heads": heads, "slots": slots, "far": far, "head_dim": head_dim, "rotary": rotary or head_dim,
            "layout": layout, "dtype": dtype, "scaling": scaling, "factor": factor, "backward": backward}


def _append(name, batch, longest, most, rotate=False, layout="half", store="e4m3", page=64, heads=32, kv_heads=8, head_dim=128, dtype="fp16", mix=0):
    return {"name": name, "op": "append", "batch": batch, "longest": longest, "most": most, "rotate": rotate, "layout": layout, "store": store,
            "page": page, "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim, "dtype": dtype, "idle": 0, "mix": mix}


def _read(name, batch, longest, store="e4m3", page=64, kv_heads=8, head_dim=128, dtype="fp16", mix=0):
    return {"name": name, "op": "read", "batch": batch, "longest": longest, "most": longest, "store": store, "page": page, "kv_heads": kv_heads,
            "head_dim": head_dim, "dtype": dtype, "idle": 0, "mix": mix}


def _attend(name, batch, longest, most=1, heads=32, kv_heads=8, head_dim=128, store="e4m3", page=64, dtype="fp16", window=0, idle=0, lse=False, mix=0):
    return {"name": name, "op": "attend", "batch": batch, "longest": longest, "most": most, "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim,
            "store": store, "page": page, "dtype": dtype, "window": window, "idle": idle, "lse": lse, "mix": mix}


def _lengths(case):
    """(new, total) tokens of each sequence: the first has the most of both, the last `idle` ones none in the cache."""
    r = random.Random(case["mix"])
    b, most, longest = case["batch"], case["most"], case["longest"]
    new = [most] + [r.randint(max(1, most // 4), most) for _ in range(b - 1)]
    total = [longest] + [n + int((longest - most) * r.uniform(0.2, 1.0)) for n in new[1:]]
    return new, [0 if i >= b - case["idle"] else t for i, t in enumerate(total)]


def work(case):
    if case["op"] == "rope":
        n = case["tokens"] * case["heads"] * case["head_dim"]
        return {"bytes": 4 * n + 4 * case["tokens"] + 4 * case["rotary"], "flops": 3 * case["tokens"] * case["heads"] * case["rotary"]}
    new, total = _lengths(case)
    row, page = case["kv_heads"] * case["head_dim"], case["page"]
    if case["op"] == "append":
        n = sum(new)
        touched = sum((t + page - 1) // page - (t - k) // page for k, t in zip(new, total))
        nbytes = n * row * 2 * 3 + touched * case["kv_heads"] * 8 + touched * 4
        if case["rotate"]:
            nbytes += n * case["heads"] * case["head_dim"] * 4 + 4 * case["head_dim"]
        return {"bytes": nbytes, "flops": 4 * n * row}
    if case["op"] == "read":
        n = sum(new)
        return {"bytes": n * row * 2 * 3 + sum((t + page - 1) // page for t in new) * (case["kv_heads"] * 8 + 4), "flops": 2 * n * row}
    seen = pairs = 0
    for n, t in zip(new, total):
        w = case["window"] or t + n
        first = max(0, t - n - w + 1)
        seen += max(0, t - first)
        full = [min(w, p + 1) for p in range(max(0, t - n), t)]
        pairs += sum(full)
    heads = case["heads"] * case["head_dim"]
    nbytes = seen * row * 2 + (seen + page - 1) // page * (case["kv_heads"] * 8 + 4) + sum(new) * heads * 4
    if case["lse"]:
        nbytes += sum(new) * case["heads"] * 4
    return {"bytes": nbytes, "flops": 4 * pairs * heads}


# ---------------------------------------------------------------- inputs

def _frequencies(case, dev):
    """Radians per position of each rotated pair, in 64 bits, and the factor that the rotated values get."""
    d, base, length = case.get("rotary") or case["head_dim"], 10000.0, 4096
    kind, factor = case.get("scaling", "none"), case.get("factor", 1.0)
    if kind == "ntk":
        base *= factor ** (d / (d - 2))
    i = torch.arange(0, d, 2, dtype=torch.float64)
    freq = base ** (-i / d)
    amplitude = 1.0
    if kind == "linear":
        freq = freq / factor
    elif kind == "yarn":  # pairs that turn often within the trained length stay, slow ones are stretched, a ramp between
        def pair(turns):
            return d * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(base))
        low, high = max(math.floor(pair(32)), 0), min(math.ceil(pair(1)), d - 1)
        keep = 1 - ((torch.arange(d // 2, dtype=torch.float64) - low) / max(high - low, 0.001)).clamp(0, 1)
        freq = freq * keep + freq / factor * (1 - keep)
        amplitude = 0.1 * math.log(factor) + 1.0
    return freq.to(dev), amplitude


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    half = HALF[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=half)

    s = {"case": case}
    if case["op"] == "rope":
        s["x"] = normal(case["tokens"], case["slots"], case["head_dim"])[:, :case["heads"]]
        first = int(torch.randint(0, max(1, case["far"] - case["tokens"] + 2), (1,), generator=g, device=dev))
        s["pos"] = torch.arange(first, first + case["tokens"], device=dev, dtype=torch.int32)
        s["freq"], s["amplitude"] = _frequencies(case, dev)
        return s
    new, total = _lengths(case)
    kv, dim, page, batch = case["kv_heads"], case["head_dim"], case["page"], case["batch"]
    width = max(-(-max(total) // page), 1)
    need = torch.tensor([-(-t // page) for t in total])
    pages = int(need.sum()) + 8
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    start = (need.cumsum(0) - need).to(dev)
    at = (start[:, None] + torch.arange(width, device=dev)).clamp(max=pages - 1)
    # entries past a sequence's last page are never looked at
    s["table"] = torch.where(torch.arange(width, device=dev) < need.to(dev)[:, None], order[at], -1)

    def codes():
        if case["store"] == "int8":
            return torch.randint(-127, 128, (pages, kv, page, dim), generator=g, device=dev, dtype=torch.int8)
        return torch.cat([(torch.randn(n, kv, page, dim, generator=g, device=dev, dtype=torch.float16) * 110).clamp(-448, 448).to(torch.float8_e4m3fn)
                          .view(torch.uint8) for n in [4096] * (pages // 4096) + [pages % 4096]]).view(torch.float8_e4m3fn)

    def scales():  # of values whose root mean square is near 1, from block to block up to a factor of 2 apart
        mid = 1 / 73.6 if case["store"] == "int8" else 1 / 110
        return torch.rand(pages, kv, generator=g, device=dev).mul(2).sub(1).exp2().mul(mid)

    s["k"], s["v"], s["ks"], s["vs"] = codes(), codes(), scales(), scales()
    s["cu"] = torch.tensor([0] + new, device=dev).cumsum(0).to(torch.int32)
    s["most"], s["longest"] = case["most"], case["longest"]
    if case["op"] == "attend":
        s["lens"] = torch.tensor(total, device=dev, dtype=torch.int32)
        s["q"] = normal(sum(new), case["heads"], dim) * 1.5
    elif case["op"] == "read":
        s["first"] = torch.zeros(batch, device=dev, dtype=torch.int32)
        s["tokens"] = sum(new)
    else:
        s["lens"] = torch.tensor([t - n for n, t in zip(new, total)], device=dev, dtype=torch.int32)
        spread = torch.rand(kv, dim, generator=g, device=dev).mul(2).sub(1).exp2().to(half)  # some channels are larger than others
        s["new_k"], s["new_v"] = normal(sum(new), kv, dim) * spread, normal(sum(new), kv, dim)
        if case["rotate"]:
            s["q"] = normal(sum(new), case["heads"], dim)
            s["freq"], s["amplitude"] = _frequencies(case, dev)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    case = s["case"]
    if own:
        import tiled_tensor_core_tcgen05_gb300 as tg
        layout = tg.ROPE_INTERLEAVED if case.get("layout") == "interleaved" else tg.ROPE_HALF
        if case["op"] == "rope":
            return tg.rope(s["x"], s["pos"], s["freq"], s["amplitude"], layout=layout, backward=case["backward"])
        cache = tg.KvCache(s["k"], s["v"], s["ks"], s["vs"])
        if case["op"] == "append":
            if case["rotate"]:
                q = tg.kv_append(cache, s["new_k"], s["new_v"], s["table"], s["lens"], s["cu"], max_new=s["most"], Q=s["q"], inv_freq=s["freq"],
                                 amplitude=s["amplitude"], layout=layout)
                return [s["k"], s["v"], s["ks"], s["vs"], q]
            tg.kv_append(cache, s["new_k"], s["new_v"], s["table"], s["lens"], s["cu"], max_new=s["most"])
            return [s["k"], s["v"], s["ks"], s["vs"]]
        if case["op"] == "read":
            return tg.kv_read(cache, s["table"], s["first"], s["cu"], s["tokens"], dtype=HALF[case["dtype"]])
        return tg.attention_kv(s["q"], cache, s["table"], s["lens"], s["cu"], max_new=s["most"], max_len=s["longest"], window=case["window"],
                               return_lse=case["lse"])
    if case["op"] == "rope":
        return _rotate(s["x"].float(), s["pos"], s["freq"], s["amplitude"], case["layout"], -1.0 if case["backward"] else 1.0).to(s["x"].dtype)
    if case["op"] == "append":
        return _write(s)
    if case["op"] == "read":
        return _back(s)
    return _attention(s)


def _rotate(x, pos, freq, amplitude, layout, sign):
    """x (tokens, heads, dim) in 32 bits; the first 2 * len(freq) values of each head are turned in pairs, the others stay."""
    angle = pos.double()[:, None] * freq
    c, d = (angle.cos() * amplitude).float()[:, None], (angle.sin() * (sign * amplitude)).float()[:, None]
    n = 2 * freq.numel()
    if layout == "half":
        a, b = x[..., :n // 2], x[..., n // 2:n]
        turned = torch.cat([a * c - b * d, b * c + a * d], -1)
    else:
        a, b = x[..., 0:n:2], x[..., 1:n:2]
        turned = torch.stack([a * c - b * d, b * c + a * d], -1).flatten(-2)
    return torch.cat([turned, x[..., n:]], -1)


def _of_tokens(s, first, tokens):
    """The sequence, the place in it, the page and the place in the page of each packed token; sequence i's begin at first[i]."""
    t = torch.arange(tokens, device=s["cu"].device)
    b = torch.searchsorted(s["cu"][1:].contiguous(), t.to(torch.int32), right=True)
    pos = first[b] + t - s["cu"][b]
    return b, pos, s["table"][b, pos // s["case"]["page"]].long(), pos % s["case"]["page"]


def _code(x, store):
    """x in units of its block's scale, rounded to nearest even into the store's type."""
    return x.round().clamp(-127, 127).to(torch.int8) if store == "int8" else x.clamp(-448, 448).to(torch.float8_e4m3fn)


def _bytes(codes):
    return codes.view(torch.uint8)


def _write(s):
    case = s["case"]
    store, page, kv = case["store"], case["page"], case["kv_heads"]
    b, pos, at, place = _of_tokens(s, s["lens"], s["new_k"].shape[0])
    k, v = s["new_k"].float(), s["new_v"].float()
    outputs = []
    if case["rotate"]:
        k = _rotate(k, pos, s["freq"], s["amplitude"], case["layout"], 1.0)
        outputs = [_rotate(s["q"].float(), pos, s["freq"], s["amplitude"], case["layout"], 1.0).to(s["q"].dtype)]
    begun = (place == 0)
    # the pages that are partly filled: each sequence's last one before the call
    some = (s["lens"] % page > 0) & (s["cu"][1:] > s["cu"][:-1])
    old = s["table"].gather(1, (s["lens"] // page).long().clamp(max=s["table"].shape[1] - 1)[:, None])[:, 0].long()[some]
    held = (torch.arange(page, device=b.device) < (s["lens"] % page)[some][:, None])[:, None, :, None]

    def one(x, codes, scales):
        most = torch.zeros_like(scales).scatter_reduce_(0, at[:, None].expand(-1, kv), x.abs().amax(-1), "amax")
        fresh = torch.zeros(scales.shape[0], dtype=torch.bool, device=b.device).index_fill_(0, at[begun], True)
        touched = torch.zeros_like(fresh).index_fill_(0, at, True)
        before = torch.where(fresh[:, None], 0.0, scales)
        after = torch.where(touched[:, None], torch.maximum(before, (most / QMAX[store]).clamp(min=FLOOR)), scales)
        per = 1.0 / after
        ratio = (before * per)[old][:, :, None, None]
        again = _code(codes[old].float() * ratio, store)
        _bytes(codes)[old] = torch.where(held, _bytes(again), _bytes(codes)[old])
        _bytes(codes)[at, :, place] = _bytes(_code(x * per[at][..., None], store))
        scales.copy_(after)

    one(k, s["k"], s["ks"])
    one(v, s["v"], s["vs"])
    return [s["k"], s["v"], s["ks"], s["vs"]] + outputs


def _back(s):
    _, _, at, place = _of_tokens(s, s["first"], s["tokens"])
    half = HALF[s["case"]["dtype"]]
    return [((_bytes(c)[at, :, place]).view(c.dtype).float() * f[at][..., None]).to(half) for c, f in ((s["k"], s["ks"]), (s["v"], s["vs"]))]


def _dense(codes, scales, at, kv, dim):
    """(batch, kv, tokens, dim) in 32 bits of the pages `at` (batch, n)."""
    x = _bytes(codes)[at].view(codes.dtype).float() * scales[at][..., None, None]
    return x.transpose(1, 2).reshape(at.shape[0], kv, -1, dim)


def _attention(s):
    case = s["case"]
    kv, dim, page, share = case["kv_heads"], case["head_dim"], case["page"], case["heads"] // case["kv_heads"]
    batch, most = case["batch"], s["most"]
    dev = s["q"].device
    at = s["table"].long().clamp(min=0)
    new = (s["cu"][1:] - s["cu"][:-1]).long()
    rows = (s["cu"][:-1].long()[:, None] + torch.arange(most, device=dev)).clamp(max=s["q"].shape[0] - 1)
    q = s["q"].float()[rows].view(batch, most, kv, share, dim).permute(0, 2, 3, 1, 4).reshape(batch, kv, share * most, dim)
    k = _dense(s["k"], s["ks"], at, kv, dim)
    score = q @ k.transpose(-1, -2) / math.sqrt(dim)
    del k
    here = (s["lens"].long() - new)[:, None] + torch.arange(most, device=dev)
    key = torch.arange(score.shape[-1], device=dev)
    seen = (key <= here[..., None]) & (key < s["lens"][:, None, None])
    if case["window"]:
        seen &= key > here[..., None] - case["window"]
    score = score.view(batch, kv, share, most, -1).masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = (score - torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    v = _dense(s["v"], s["vs"], at, kv, dim)
    v = v.masked_fill_((key >= s["lens"][:, None])[:, None, :, None], 0.0)
    o = (p.view(batch, kv, share * most, -1) @ v).view(batch, kv, share, most, dim) / torch.where(total == 0, 1.0, total)
    t = torch.arange(s["q"].shape[0], device=dev)
    b = torch.searchsorted(s["cu"][1:].contiguous(), t.to(torch.int32), right=True)
    j = t - s["cu"][b]
    out = o[b, :, :, j].reshape(-1, case["heads"], dim).to(s["q"].dtype)
    if not case["lse"]:
        return out
    return [out, (top + total.log())[b, :, :, j].reshape(-1, case["heads"])]


# ---------------------------------------------------------------- the definitions, in 64 bits

def _turn64(x, pos, freq, amplitude, layout, backward):
    """Multiplication of each pair, as a complex number, by amplitude * exp(+-i pos freq)."""
    x = x.double().clone()
    n = 2 * freq.numel()
    z = torch.polar(torch.full_like(freq, amplitude).expand(pos.numel(), -1).contiguous(), (pos.double()[:, None] * freq) * (-1.0 if backward else 1.0))
    first, second = (slice(0, n // 2), slice(n // 2, n)) if layout == "half" else (slice(0, n, 2), slice(1, n, 2))
    w = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * z[:, None]
    x[..., first], x[..., second] = w.real, w.imag
    return x


def _grid64(x):
    """x rounded to the nearest e4m3 value, ties to the even one: steps of 2^(e - 3) from 2^e on, of 2^-9 below 2^-6."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 1).clamp(min=-6) - 3)
    return (x / step).round().mul(step).clamp(-448, 448)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _turn64(s["x"], s["pos"], s["freq"], s["amplitude"], case["layout"], case["backward"])
    new, total = _lengths(case)
    page, kv, dim = case["page"], case["kv_heads"], case["head_dim"]
    table, store = s["table"].long(), case["store"]
    if case["op"] == "append":
        if store == "int8":
            return None
        k, v, q = s["new_k"].double(), s["new_v"].double(), None
        if case["rotate"]:
            where = torch.cat([torch.arange(t - n, t, device=k.device) for n, t in zip(new, total)])
            k, q = (_turn64(x, where, s["freq"], s["amplitude"], case["layout"], False) for x in (s["new_k"], s["q"]))
        found = []
        for x, codes, scales in ((k, s["k"].double(), s["ks"].double()), (v, s["v"].double(), s["vs"].double())):
            done = 0
            for i, (n, t) in enumerate(zip(new, total)):
                place = t - n
                while place < t:
                    many = min(page - place % page, t - place)
                    p, o = table[i, place // page], place % page
                    rows = x[done:done + many]
                    scale = (rows.abs().amax((0, 2)) / QMAX[store]).clamp(min=FLOOR)
                    if o:
                        scale = torch.maximum(scale, scales[p])
                        codes[p, :, :o] = _grid64(codes[p, :, :o] * (scales[p] / scale)[:, None, None])
                    codes[p, :, o:o + many] = _grid64(rows / scale[:, None]).transpose(0, 1)
                    scales[p] = scale
                    place, done = place + many, done + many
            found.append((codes, scales))
        out = [found[0][0], found[1][0], found[0][1], found[1][1]]
        return out + [q] if case["rotate"] else out
    if case["op"] == "read":
        found = []
        for codes, scales in ((s["k"], s["ks"]), (s["v"], s["vs"])):
            parts = []
            for i, n in enumerate(new):
                use = table[i, :-(-n // page)]
                x = codes.view(torch.uint8)[use].view(codes.dtype).double() * scales[use].double()[:, :, None, None]
                parts.append(x.permute(0, 2, 1, 3).reshape(-1, kv, dim)[:n])
            found.append(torch.cat(parts))
        return found
    if work(case)["flops"] > 4e12:
        return None
    out, lse, done = [], [], 0
    for i, (n, t) in enumerate(zip(new, total)):
        q = s["q"][done:done + n].double().view(n, kv, -1, dim)
        done += n
        use = table[i, :-(-t // page)]
        k, v = ((c.view(torch.uint8)[use].view(c.dtype).double() * f[use].double()[:, :, None, None]).transpose(0, 1).reshape(kv, -1, dim)[:, :t]
                for c, f in ((s["k"], s["ks"]), (s["v"], s["vs"])))
        rel = torch.arange(t - n, t, device=q.device)[:, None] - torch.arange(t, device=q.device)
        hidden = rel < 0 if not case["window"] else (rel < 0) | (rel >= case["window"])
        o, l = torch.zeros_like(q), torch.full(q.shape[:3], -math.inf, dtype=torch.float64, device=q.device)
        for h in range(kv if t else 0):
            for j in range(q.shape[2]):
                z = (q[:, h, j] @ k[h].T / math.sqrt(dim)).masked_fill(hidden, -math.inf)
                l[:, h, j] = torch.logsumexp(z, -1)
                o[:, h, j] = (z - l[:, h, j][:, None]).exp().nan_to_num(0.0) @ v[h]
        out.append(o.reshape(n, -1, dim))
        lse.append(l.reshape(n, -1))
    return [torch.cat(out), torch.cat(lse)] if case["lse"] else torch.cat(out)
